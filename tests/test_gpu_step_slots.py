"""GPU parity of gdr_step_slots (the recurrent form over a pool of state slots)
against the fp64 oracle, on the very values the kernel reads.

Tolerances (max|d| / max|ref|), worst case per token: a row's dot product adds
dk / 8 products per lane in sequence, then 3 sums, with about 4 more roundings
(gate, normalisation, erase, write): (dk / 8 + 7) 2^-24 of sum |S_j k_j| <= |S_i| |k|
<= sqrt(dk) max|S| for a unit key, and the errors of the tokens add up since
every transition is a contraction.  exp, log1p, rsqrt are within 4 ulp.  A bf16 o is
rounded once more, by at most 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import SLOT_SKIP, SLOT_ZERO, binding
from oracle import layer

pytestmark = pytest.mark.gpu


def tolerance(dk, tokens, dtype=torch.float32):
    fp32 = (tokens + 1) * (dk / 8 + 7 + 8) * 2.0**-24 * dk**0.5
    return fp32 + (2.0**-8 if dtype == torch.bfloat16 else 0.0)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(lens, Hk, H, dk, dv, dtype, gate="scalar", raw=False, fused=False, slots=None, seed=0,
         dev="cuda"):
    """A batch of requests with the pool they live in (every slot filled)."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    total = sum(lens)
    width = [Hk * dk, Hk * dk, H * dv]
    rows = n(total, sum(width))
    if not raw:
        for i in range(2):
            part = rows[:, i * Hk * dk:(i + 1) * Hk * dk].view(total, Hk, dk)
            part /= part.norm(dim=-1, keepdim=True).clamp_min(1e-12)
    rows = rows.to(dtype).to(dev)
    parts = rows.split(width, dim=1)
    q, k, v = ((p if fused else p.contiguous()).unflatten(1, s)
               for p, s in zip(parts, ((Hk, dk), (Hk, dk), (H, dv))))
    g = n(total, H, dk) if gate == "channel" else n(total, H)
    beta = n(total, H)
    scale = 0.05 + 0.1 * torch.rand(H, generator=gen) if raw else None
    if not raw:
        g, beta = -0.1 * torch.nn.functional.softplus(g), torch.sigmoid(beta)
    pool = 0.3 * n(slots or len(lens) + 2, H, dv, dk)
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32)
    d = dict(q=q, k=k, v=v, g=g.to(dev), beta=beta.to(dev), pool=pool.to(dev), cu=cu.to(dev),
             scale=None if scale is None else scale.to(dev), raw=raw)
    return d


def i32(x, dev="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def call(d, src, dst=None, cu=True, **kw):
    return binding.step_slots(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], src, dst=dst,
                              cu_seqlens=d["cu"] if cu else None, gate_scale=d["scale"],
                              norm_q=d["raw"], norm_k=d["raw"], **kw)


def expect(d, src, dst=None, cu=True, o=None):
    return layer.step_slots(f64(d["q"]), f64(d["k"]), f64(d["v"]), f64(d["g"]), f64(d["beta"]),
                            f64(d["pool"]), src.tolist(), None if dst is None else dst.tolist(),
                            d["cu"].tolist() if cu else None, f64(d["scale"]), d["raw"], d["raw"],
                            None if o is None else f64(o))


def close(got, want, tol, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    e = np.abs(got - want).max() / max(np.abs(want).max(), 1e-30)
    assert e <= tol, f"{what}: {e:.3e} > {tol:.3e}"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 64), (128, 128), (32, 128)])
@pytest.mark.parametrize("raw", [True, False])
def test_one_token_in_place(cuda_device, dtype, gate, dk, dv, raw):
    """The decode step: a token a request, the state updated in its slot."""
    d = make([1] * 5, 2, 6, dk, dv, dtype, gate, raw, fused=raw, slots=9, seed=dk + dv)
    src = i32([7, 0, 3, 8, 2])
    ro, rp = expect(d, src, cu=False)
    o = call(d, src, cu=False)
    torch.cuda.synchronize()
    close(o, ro, tolerance(dk, 1, dtype), "o")
    close(d["pool"], rp, tolerance(dk, 1), "pool")
    untouched = [1, 4, 5, 6]
    assert np.array_equal(f64(d["pool"])[untouched], rp[untouched])


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_many_small_states(cuda_device, gate, dv):
    """Keys of 32 channels and more rows than the one-token kernel takes: the same
    step through the other kernel, skipped and new requests among them."""
    R, H = 16384 // (4 * dv) + 3, 4
    d = make([1] * R, 2, H, 32, dv, torch.bfloat16, gate, True, slots=R + 5, seed=dv)
    src = torch.randperm(R + 5, generator=torch.Generator().manual_seed(1))[:R].int().cuda()
    src[3], src[7] = SLOT_SKIP, SLOT_ZERO
    o = torch.full_like(d["v"], 3.0)
    ro, rp = expect(d, src, cu=False, o=o)
    call(d, src, cu=False, o=o)
    torch.cuda.synchronize()
    assert binding.device_status() == 0 and (o[3] == 3.0).all()
    close(o, ro, tolerance(32, 1, torch.bfloat16), "o")
    close(d["pool"], rp, tolerance(32, 1), "pool")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("fused", [True, False])
def test_ragged_requests_keep_every_state(cuda_device, dtype, gate, fused):
    """1 to 9 tokens a request (over the 4 that are prepared at a time), no token
    at all, a new request, the state kept after each token."""
    lens = [3, 1, 0, 9, 4, 5, 2]
    d = make(lens, 2, 4, 128, 128, dtype, gate, True, fused, slots=40, seed=5)
    perm = np.random.default_rng(5).permutation(40)
    dst = i32(perm[:24])
    # request 3 starts from one of the slots it writes, request 4 is new, 2 has no tokens
    src = i32([perm[30], perm[31], perm[32], perm[4], SLOT_ZERO, perm[33], perm[34]])
    ro, rp = expect(d, src, dst)
    o = call(d, src, dst)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    close(o, ro, tolerance(128, 9, dtype), "o")
    close(d["pool"], rp, tolerance(128, 9), "pool")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_head_dims_with_several_tokens(cuda_device, dtype, gate, dk, dv):
    """Every head size, three value heads to a key head, over the 8 tokens that are
    prepared at a time."""
    lens = [2, 11, 1]
    d = make(lens, 1, 3, dk, dv, dtype, gate, True, seed=dk * dv, slots=16)
    src, dst = i32([15, SLOT_ZERO, 1]), i32([0, 2, *[-1] * 9, 3, 4, 5])
    ro, rp = expect(d, src, dst)
    o = call(d, src, dst)
    torch.cuda.synchronize()
    close(o, ro, tolerance(dk, 11, dtype), "o")
    close(d["pool"], rp, tolerance(dk, 11), "pool")


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("cu", [True, False])
def test_nan_and_infinities_stay_with_their_request(cuda_device, gate, cu):
    """A NaN key, an infinite value and a slot full of NaN reach their own request's
    output and state only; a new request does not read what its slot held."""
    d = make([1] * 4, 1, 2, 64, 64, torch.float32, gate, slots=8, seed=21)
    src, dst = i32([0, 1, 2, SLOT_ZERO]), i32([0, 1, 2, 3])
    clean = dict(d, pool=d["pool"].clone())
    want = call(clean, src, dst, cu=cu)
    d["k"][0], d["v"][1], d["pool"][2], d["pool"][3] = (float("nan"), float("inf"), float("nan"),
                                                        float("nan"))
    o = call(d, src, dst, cu=cu)
    torch.cuda.synchronize()
    assert torch.isnan(o[0]).all() and not torch.isfinite(o[1]).all() and torch.isnan(o[2]).all()
    assert torch.equal(o[3], want[3]) and torch.equal(d["pool"][3:], clean["pool"][3:])


@pytest.mark.parametrize("tokens", [1, 4, 5, 301])
def test_long_requests_without_dst(cuda_device, tokens):
    """dst None: the last state goes back to the slot it came from."""
    d = make([tokens, 1], 1, 1, 64, 64, torch.float32, seed=tokens)
    src = i32([1, 3])
    ro, rp = expect(d, src)
    o = call(d, src)
    torch.cuda.synchronize()
    close(o, ro, tolerance(64, tokens), "o")
    close(d["pool"], rp, tolerance(64, tokens), "pool")


def test_equals_the_dense_step(cuda_device):
    """The same states as gdr_step updates, addressed by slot: equal to within
    fp32 roundings (the sums run in another order)."""
    d = make([1] * 6, 4, 4, 128, 128, torch.bfloat16, slots=6, seed=9)
    S = d["pool"].clone()
    o1 = binding.step(d["q"], d["k"], d["v"], d["g"], d["beta"], S)
    o2 = call(d, i32(range(6)), cu=False)
    torch.cuda.synchronize()
    close(o2, f64(o1), tolerance(128, 1) + 2.0**-7, "o")
    close(d["pool"], f64(S), 2 * tolerance(128, 1), "pool")


def test_prefill_then_pooled_decode(cuda_device):
    """gdr_chunk_fwd_varlen's final states, put into slots, go on as if the
    sequence had never been cut."""
    lens, more = [70, 1, 130], 3
    d = make([n + more for n in lens], 2, 2, 64, 64, torch.float32, seed=10)
    cu = d["cu"].tolist()
    first = torch.cat([torch.arange(cu[i], cu[i] + n) for i, n in enumerate(lens)]).cuda()
    rest = torch.cat([torch.arange(cu[i] + n, cu[i + 1]) for i, n in enumerate(lens)]).cuda()
    slots = i32([4, 0, 2])
    whole, _ = layer.step_slots(*(f64(d[n]) for n in ("q", "k", "v", "g", "beta")),
                                np.zeros(d["pool"].shape), [-1] * 3, cu=cu)
    pick = lambda idx: [d[n][idx].contiguous() for n in ("q", "k", "v", "g", "beta")]
    o1, S = binding.chunk_fwd_varlen(*pick(first), i32([0, 70, 71, 201]))
    d["pool"][slots.long()] = S
    o2 = binding.step_slots(*pick(rest), d["pool"], slots, cu_seqlens=i32([0, 3, 6, 9]))
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    # (the chunked forward's own bar for fp32 inputs is 1e-4)
    close(o1, whole[first.cpu().numpy()], 1e-4, "prefill o")
    close(o2, whole[rest.cpu().numpy()], 1e-4 + tolerance(64, more), "decode o")


def test_forks_share_a_start(cuda_device):
    """Requests that only read a slot may share it; each keeps its own branch."""
    d = make([2, 2, 1], 1, 2, 64, 64, torch.float32, slots=8, seed=11)
    src, dst = i32([5, 5, 5]), i32([-1, 0, 1, 2, 3])
    ro, rp = expect(d, src, dst)
    o = call(d, src, dst)
    torch.cuda.synchronize()
    close(o, ro, tolerance(64, 2), "o")
    close(d["pool"], rp, tolerance(64, 2), "pool")


def test_one_slot_named_twice_by_a_request(cuda_device):
    """The last write stays."""
    d = make([6], 1, 1, 32, 32, torch.float32, slots=3, seed=12)
    src, dst = i32([1]), i32([1, 2, 1, 2, 1, -1])
    ro, rp = expect(d, src, dst)
    o = call(d, src, dst)
    torch.cuda.synchronize()
    close(o, ro, tolerance(32, 6), "o")
    close(d["pool"], rp, tolerance(32, 6), "pool")


def test_rows_of_nobody_stay(cuda_device):
    """Skipped requests, rows behind the last sequence and slots outside the pool:
    o and the pool stay as they were there, bit for bit; only the last two are recorded."""
    assert binding.device_status() == 0
    d = make([2, 1, 3, 1, 2, 4], 1, 2, 64, 64, torch.bfloat16, slots=7, seed=13)
    d["pool"][6] = float("nan")  # never read
    d["cu"] = i32([0, 2, 3, 6, 7, 9, 9])  # the last four rows are padding
    o = torch.full((13, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    dst = i32([0, 0, 1, 2, 2, 2, 3, 4, 4] + [6] * 4)
    for bad, status in ((SLOT_SKIP, 0), (7, binding.GDR_ERR_SLOT), (-3, binding.GDR_ERR_SLOT),
                        (2**31 - 1, binding.GDR_ERR_SLOT)):
        src = i32([0, bad, 2, SLOT_ZERO, 4, 6])
        o.fill_(7.0)
        ro, rp = expect(d, src, dst, o=o)
        pool = d["pool"].clone()
        call(d, src, dst, o=o)
        torch.cuda.synchronize()
        assert binding.device_status() == status
        close(o, ro, tolerance(64, 3, torch.bfloat16), "o")
        assert torch.equal(o[[2, 9, 10, 11, 12]], torch.full_like(o[:5], 7.0))
        assert torch.equal(d["pool"][[1, 5]], pool[[1, 5]])
        close(d["pool"][:6], rp[:6], tolerance(64, 3), "pool")
    # a dst outside the pool is not written, its tokens run all the same
    dst2 = i32([0, 9, 1, 2, 2, -2, 3, 4, 4] + [6] * 4)
    src = i32([0, 1, 2, 3, 4, 6])
    ro, rp = expect(d, src, dst2, o=o)
    call(d, src, dst2, o=o)
    torch.cuda.synchronize()
    assert binding.device_status() == binding.GDR_ERR_SLOT
    close(o, ro, tolerance(64, 3, torch.bfloat16), "o")
    close(d["pool"][:6], rp[:6], tolerance(64, 3), "pool")


def test_bad_offsets_are_clamped(cuda_device):
    """cu_seqlens outside [0, total] or falling: nothing out of range is read."""
    d = make([2, 2, 2], 1, 1, 32, 32, torch.float32, slots=4, seed=14)
    d["cu"] = i32([-5, 2, 1, 99])
    src = i32([0, 1, 2])
    o = call(d, src, o=torch.zeros_like(d["v"]))
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    # (tokens 0-1 of request 0, none of request 1, tokens 1-5 of request 2)
    assert torch.isfinite(o).all() and torch.isfinite(d["pool"]).all()


@pytest.mark.parametrize("g", [-30.0, -1e4, 0.0])
def test_extreme_gates_and_strengths(cuda_device, g):
    """alpha from nearly nothing to one; beta 0 and 1."""
    d = make([3, 3], 1, 2, 64, 64, torch.float32, seed=15)
    d["g"].fill_(g)
    d["beta"][::2] = 0.0
    d["beta"][1::2] = 1.0
    src = i32([0, 2])
    ro, rp = expect(d, src)
    o = call(d, src)
    torch.cuda.synchronize()
    close(o, ro, tolerance(64, 3), "o")
    close(d["pool"], rp, tolerance(64, 3), "pool")


def test_raw_logits_far_out_and_zero_rows(cuda_device):
    """Logits of +-200, an all-zero key (it stays zero: nothing is written)."""
    d = make([4], 1, 2, 64, 32, torch.float32, raw=True, slots=2, seed=16)
    d["g"][0], d["g"][1], d["beta"][2], d["beta"][3] = 200.0, -200.0, 200.0, -200.0
    d["k"][1] = 0.0
    src = i32([1])
    ro, rp = expect(d, src)
    o = call(d, src)
    torch.cuda.synchronize()
    close(o, ro, tolerance(64, 4), "o")
    close(d["pool"], rp, tolerance(64, 4), "pool")


def test_pool_slots_apart_and_far(cuda_device):
    """Slots with room between them, the last one more than 2^32 bytes (and 2^31
    elements) behind the first."""
    H, dv, dk = 1, 128, 128
    apart = 1 << 20
    slots = (1 << 31) // apart + 3
    whole = torch.empty(slots * apart, dtype=torch.float32, device="cuda")
    pool = whole.view(slots, apart)[:, : H * dv * dk].view(slots, H, dv, dk)
    d = make([1, 2], 1, H, dk, dv, torch.bfloat16, seed=17)
    start = d["pool"].clone()
    pool[slots - 1], pool[0] = start[0], start[1]
    src = i32([0, 1])
    ro, rp = expect(d, src)
    whole[H * dv * dk:apart] = 5.0
    d["pool"] = pool
    o = call(d, i32([slots - 1, 0]))
    torch.cuda.synchronize()
    close(o, ro, tolerance(dk, 2, torch.bfloat16), "o")
    close(pool[slots - 1], rp[0], tolerance(dk, 2), "last slot")
    close(pool[0], rp[1], tolerance(dk, 2), "first slot")
    assert (whole[H * dv * dk:apart] == 5.0).all()


def test_other_stream_and_graph(cuda_device):
    """On a side stream, and captured once and replayed on the state it left."""
    d = make([2, 1], 1, 2, 64, 64, torch.float32, seed=18)
    src = i32([1, 3])
    steps = 3
    want = {k: v for k, v in d.items()}
    outs = []
    for _ in range(steps):
        ro, rp = expect(want, src)
        want = dict(want, pool=torch.from_numpy(rp))
        outs.append(ro)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = call(d, src, stream=side)
    side.synchronize()
    close(o, outs[0], tolerance(64, 2), "side stream o")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call(d, src)
    for i in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        close(o, outs[i], tolerance(64, 2 * (i + 1)), f"replay {i} o")
    close(d["pool"], rp, tolerance(64, 2 * steps), "pool")


def test_the_same_call_gives_the_same_bits(cuda_device):
    d = make([5, 1, 3], 2, 4, 128, 128, torch.bfloat16, "channel", True, True, slots=5, seed=19)
    runs = []
    for _ in range(2):
        e = dict(d, pool=d["pool"].clone())
        runs.append((call(e, i32([0, 1, 4])), e["pool"]))
    torch.cuda.synchronize()
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_no_requests(cuda_device):
    d = make([], 1, 1, 32, 32, torch.float32, slots=2)
    pool = d["pool"].clone()
    assert call(d, i32([])).shape == (0, 1, 32)
    assert call(d, i32([]), cu=False).shape == (0, 1, 32)
    torch.cuda.synchronize()
    assert torch.equal(pool, d["pool"])
