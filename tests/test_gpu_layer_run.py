"""The operators around the mixer run together, as a layer uses them."""
import numpy as np
import pytest
import torch

import oracle
from gated_delta_rule_93_b200 import binding
from oracle import layer, prologue

pytestmark = pytest.mark.gpu


def f64(t):
    return t.detach().double().cpu().numpy()


def rel(got, want):
    return np.abs(f64(got) - want).max() / np.abs(want).max()


def test_training_step(cuda_device):
    """prologue -> chunked forward -> output norm, and the gradients all the way
    back to the raw projections, against the fp64 chain (fp32 inputs: every
    link is within 1e-4 of its own oracle, the chunked forward's bar; six links)."""
    B, T, Hk, H, d = 2, 75, 1, 2, 32
    gen = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    q, k, v, z = n(B, T, Hk, d), n(B, T, Hk, d), n(B, T, H, d), n(B, T, H, d)
    a, b, dy = n(B, T, H), n(B, T, H), n(B, T, H, d)
    scale, w = (0.1 + 0.1 * torch.rand(H, generator=gen)).cuda(), 1 + 0.2 * n(d)

    raw = (q, k, a, b, scale)
    qn, kn, g, beta = binding.prologue_fwd(*raw)
    o, _ = binding.chunk_fwd(qn, kn, v, g, beta, output_final_state=False)
    y = binding.group_norm_fwd(o, z, w)
    dn = binding.group_norm_bwd(dy, o, z, w)
    dc = binding.chunk_bwd(qn, kn, v, g, beta, dn["dx"])
    dp = binding.prologue_bwd(*raw, dc["dq"], dc["dk"], dc["dg"], dc["dbeta"])
    torch.cuda.synchronize()
    assert binding.device_status() == 0

    up = lambda t: np.repeat(f64(t), H // Hk, axis=2)
    q6, k6, g6, b6 = prologue.prologue(up(q), up(k), f64(a), f64(b), f64(scale))
    c32 = lambda x: np.ascontiguousarray(x, dtype=np.float32)
    o6, _ = oracle.gdr_fwd_f64(q6, k6, f64(v), g6, b6)
    flat = lambda x: x.reshape(B * T, *x.shape[2:])
    n6 = layer.group_norm_grad(flat(f64(dy)), flat(o6), flat(f64(z)), f64(w))
    # (the backward oracle takes fp32 inputs: rounding q, k, g, beta costs 2^-24 each)
    d6 = oracle.gdr_bwd(c32(q6), c32(k6), c32(f64(v)), c32(g6), c32(b6),
                        n6["dx"].reshape(B, T, H, d))
    p6 = layer.prologue_grad(flat(f64(q)), flat(f64(k)), flat(f64(a)), flat(f64(b)), f64(scale),
                             *(flat(np.asarray(d6[x])) for x in ("dq", "dk", "dg", "dbeta")))
    tol = 6e-4
    assert rel(y.flatten(0, 1), layer.group_norm(flat(o6), flat(f64(z)), f64(w))) < tol
    for name in ("dz", "dweight"):
        got = dn[name] if name == "dweight" else dn[name].flatten(0, 1)
        assert rel(got, n6[name]) < tol, name
    assert rel(dc["dv"], np.asarray(d6["dv"])) < tol
    for name in ("dq", "dk", "da", "db", "dgate_scale"):
        got = dp[name] if name == "dgate_scale" else dp[name].flatten(0, 1)
        assert rel(got, p6[name]) < tol, name


def test_serving_steps_captured(cuda_device):
    """Slot map -> pooled decode -> output norm as one captured graph, replayed while
    the lengths and the kept counts change on the GPU: drafts checked, some
    thrown away, the state going on from the one kept."""
    R, W, Hk, H, dk, dv, room = 5, 3, 2, 4, 64, 64, 15
    gen = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    slots = R * W
    table = torch.arange(slots, dtype=torch.int32).view(R, W).flip(0).contiguous().cuda()
    pool, scale, w = torch.zeros(slots, H, dv, dk, device="cuda"), 0.1 + 0.05 * torch.rand(H, generator=gen).cuda(), 1 + 0.1 * n(dv)
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    kept = torch.zeros(R, dtype=torch.int32, device="cuda")
    width = 2 * Hk * dk + 2 * H * dv
    rows = torch.zeros(room, width, device="cuda")
    a, b = torch.zeros(room, H, device="cuda"), torch.zeros(room, H, device="cuda")
    q, k, v, z = (t.unflatten(1, s) for t, s in zip(rows.split([Hk * dk, Hk * dk, H * dv, H * dv], 1),
                                                    ((Hk, dk), (Hk, dk), (H, dv), (H, dv))))
    o = torch.zeros(room, H, dv, device="cuda")

    def step():
        m = binding.slot_map(lens, kept, table, slots, room)
        binding.step_slots(q, k, v, a, b, pool, m["src"], dst=m["dst"], cu_seqlens=m["cu_seqlens"],
                           gate_scale=scale, norm_q=True, norm_k=True, o=o)
        return m, binding.group_norm_fwd(o, z, w)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m, y = step()

    history = [[] for _ in range(R)]  # the tokens each request has kept: (q, k, v, a, b) rows
    r = np.random.default_rng(2)
    last = np.zeros(R, np.int64)  # tokens of the step before
    for turn in range(6):
        keep = np.array([r.integers(1, x + 1) if x else 0 for x in last])
        new = r.integers(1, W + 1, R)
        if turn == 3:
            new[2] = 0  # (a request pauses and goes on later from the same state)
        if turn == 4:
            keep[2] = paused
        for i in range(R):
            if turn == 4 and i == 2:
                history[2] = before_pause
            elif last[i]:
                history[i] = history[i][: len(history[i]) - int(last[i]) + int(keep[i])]
        if turn == 3:
            paused, before_pause = int(keep[2]), list(history[2])
        total = int(new.sum())
        rows.copy_(n(room, width))
        a.copy_(n(room, H))
        b.copy_(n(room, H))
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        kept.copy_(torch.tensor(keep, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        at = 0
        for i in range(R):
            tok = [tuple(f64(t[j]) for t in (q, k, v, a, b)) for j in range(at, at + int(new[i]))]
            history[i] = history[i] + tok
            if tok:
                whole = [np.stack([h[j] for h in history[i]]) for j in range(5)]
                ro, _ = layer.step_slots(*whole, np.zeros((1, H, dv, dk)), [-1], cu=[0, len(history[i])],
                                         gate_scale=f64(scale), norm_q=True, norm_k=True)
                sl = slice(at, at + len(tok))
                # fp32 all the way: (dk / 8 + 15) 2^-24 sqrt(dk) a token, the norm 16 times that of one
                assert rel(o[sl], ro[-len(tok):]) < 2e-5 * len(history[i])
                ry = layer.group_norm(ro[-len(tok):], f64(z[sl]), f64(w))
                assert rel(y[sl], ry) < 5e-4
            at += len(tok)
        assert m["cu_seqlens"].tolist()[-1] == total
        last = new
