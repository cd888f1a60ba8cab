"""GPU parity of gdr_prologue_fwd / _bwd against the fp64 oracle.

Tolerances (max|d| / max|ref|): a row's sums add at most 8 elements a lane in
sequence and 5 lane steps, with about 20 more roundings for rsqrt, exp, log1p
and the products, and dq cancels two terms at most twice its size: 4 * 64 * 2^-24.
The sums over sharing heads add `share` more.  dgate_scale: 2^-24 per
addition in sequence (tokens / tokens in flight, 128 elements, 64 steps),
relative to the sum of the terms' sizes.  bf16 outputs are rounded once more, by at most 2^-8.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import binding
from oracle import layer, prologue

pytestmark = pytest.mark.gpu

FP32 = 4 * 64 * 2.0**-24
BF16 = 2.0**-8


def f64(t):
    return t.detach().double().cpu().numpy()


def make(tokens, Hk, H, dk, dtype, gate="scalar", apart=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)

    def rows():
        t = n(tokens, Hk * dk + apart).to(dtype).cuda()
        return t[:, : Hk * dk].unflatten(1, (Hk, dk)) if apart else t.view(tokens, Hk, dk)

    a = n(tokens, H, dk) if gate == "channel" else n(tokens, H)
    return dict(q=rows(), k=rows(), a=a.cuda(), b=n(tokens, H).cuda(),
                scale=(0.05 + 0.2 * torch.rand(H, generator=gen)).cuda(),
                dq=n(tokens, H, dk).cuda(), dk=n(tokens, H, dk).cuda(),
                dg=n(*a.shape).cuda(), dbeta=n(tokens, H).cuda())


RAW, UP = ("q", "k", "a", "b", "scale"), ("dq", "dk", "dg", "dbeta")


def close(got, want, tol, what, scale=None):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    if got.size:
        e = np.abs(got - want).max() / max(np.abs(want).max() if scale is None else scale, 1e-30)
        assert e <= tol, f"{what}: {e:.3e} > {tol:.3e}"


def check(d, norm_q=True, norm_k=True):
    q, k, a, b, s = (f64(d[n]) for n in RAW)
    share = b.shape[1] // q.shape[1]
    low = BF16 if d["q"].dtype == torch.bfloat16 else 0.0
    out = binding.prologue_fwd(*(d[n] for n in RAW), norm_q=norm_q, norm_k=norm_k)
    got = binding.prologue_bwd(*(d[n] for n in RAW + UP), norm_q=norm_q, norm_k=norm_k)
    torch.cuda.synchronize()
    wq, wk = (np.repeat(prologue.l2_normalise(x) if f else x, share, axis=1)
              for x, f in ((q, norm_q), (k, norm_k)))
    close(out[0], wq, FP32 + low, "q")
    close(out[1], wk, FP32 + low, "k")
    close(out[2], prologue.log_decay(a[None], s)[0], FP32, "g")
    close(out[3], prologue.sigmoid(b), FP32, "beta")
    want = layer.prologue_grad(q, k, a, b, s, *(f64(d[n]) for n in UP), norm_q, norm_k)
    for name in ("dq", "dk"):
        assert got[name].dtype == d["q"].dtype
        close(got[name], want[name], FP32 + share * 2.0**-24 + low, name)
    for name in ("da", "db"):
        close(got[name], want[name], FP32, name)
    terms = np.abs(f64(d["dg"])) * prologue.softplus(a)
    size = terms.sum(tuple(i for i in range(a.ndim) if i != 1)).max() if a.size else 1.0
    close(got["dgate_scale"], want["dgate_scale"], FP32 + (len(a) / 100 + 192) * 2.0**-24,
          "dgate_scale", scale=size)
    return out, got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("Hk,H", [(1, 1), (2, 6), (3, 3), (5, 20)])
def test_heads(cuda_device, dtype, gate, dk, Hk, H):
    check(make(29, Hk, H, dk, dtype, gate, seed=dk + H))


@pytest.mark.parametrize("norm_q,norm_k", [(False, True), (True, False), (False, False)])
def test_flags(cuda_device, norm_q, norm_k):
    check(make(17, 2, 4, 64, torch.bfloat16, seed=1), norm_q, norm_k)


@pytest.mark.parametrize("tokens", [1, 2, 1000, 4099, 20000])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
def test_tokens(cuda_device, tokens, gate):
    check(make(tokens, 1, 3, 64, torch.bfloat16, gate, seed=tokens))


@pytest.mark.parametrize("H", [255, 257, 600])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
def test_many_heads(cuda_device, H, gate):
    """More heads than a block has gate slots."""
    check(make(5, 1, H, 32, torch.float32, gate, seed=H))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart_and_two_dimensions(cuda_device, dtype):
    d = make(24, 2, 4, 64, dtype, apart=40, seed=3)
    check(d)
    four = {n: t.unflatten(0, (4, 6)) if n != "scale" else t for n, t in d.items()}
    out, out1 = (binding.prologue_fwd(*(e[n] for n in RAW)) for e in (four, d))
    got, got1 = (binding.prologue_bwd(*(e[n] for n in RAW + UP)) for e in (four, d))
    torch.cuda.synchronize()
    for x, y in zip(out, out1):
        assert torch.equal(x.flatten(0, 1), y)
    for n in got:
        assert torch.equal(got[n] if n == "dgate_scale" else got[n].flatten(0, 1), got1[n])


def test_zero_rows_and_far_logits(cuda_device):
    """An all-zero key keeps a finite gradient (dk = dkn / 1e-3); logits of +-200 neither
    overflow nor leave the range."""
    d = make(8, 1, 2, 32, torch.float32, seed=4)
    d["a"][0], d["a"][1], d["b"][2], d["b"][3] = 200.0, -200.0, 200.0, -200.0
    d["k"][5] = 0.0
    check(d)


def test_equals_the_fused_prologue(cuda_device):
    """The map followed by chunk_fwd against chunk_fwd_prologue (fp32 inputs: the bar of
    the chunked forward, 1e-4, on both sides)."""
    d = make(90, 2, 2, 64, torch.float32, seed=5)
    v = torch.randn(1, 90, 2, 64, generator=torch.Generator().manual_seed(6)).cuda()
    one = {n: t[None] if n != "scale" else t for n, t in d.items()}
    q, k, g, beta = binding.prologue_fwd(*(one[n] for n in RAW))
    o, S = binding.chunk_fwd(q, k, v, g, beta)
    o1, S1 = binding.chunk_fwd_prologue(one["q"], one["k"], v, one["a"], one["b"], one["scale"])
    torch.cuda.synchronize()
    close(o, f64(o1), 2e-4, "o")
    close(S, f64(S1), 2e-4, "S_T")


def test_no_tokens(cuda_device):
    d = make(0, 1, 2, 32, torch.float32)
    out = binding.prologue_fwd(*(d[n] for n in RAW))
    got = binding.prologue_bwd(*(d[n] for n in RAW + UP))
    torch.cuda.synchronize()
    assert out[0].shape == (0, 2, 32) and not got["dgate_scale"].any()


def test_gradient_against_differences(cuda_device):
    """The kernel's own forward, differenced (coarse, as fp32 allows)."""
    d = make(2, 1, 2, 32, torch.float32, "channel", seed=7)
    got = binding.prologue_bwd(*(d[n] for n in RAW + UP))

    def loss():
        outs = binding.prologue_fwd(*(d[n] for n in RAW))
        return float(sum((o.double() * d[u].double()).sum() for o, u in zip(outs, UP)))

    for name, wrt in (("dq", "q"), ("dk", "k"), ("da", "a"), ("db", "b"), ("dgate_scale", "scale")):
        t = d[wrt]
        for at in ((0,) * t.dim(), tuple(s - 1 for s in t.shape)):
            keep = float(t[at])
            t[at] = keep + 1e-2
            up = loss()
            t[at] = keep - 1e-2
            down = loss()
            t[at] = keep
            assert abs((up - down) / 2e-2 - float(got[name][at])) < 5e-3, (name, at)


def test_same_bits_other_stream_and_graph(cuda_device):
    d = make(3000, 2, 4, 128, torch.bfloat16, "channel", seed=8)
    args = [d[n] for n in RAW + UP]
    a, b = binding.prologue_bwd(*args), binding.prologue_bwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = binding.prologue_bwd(*args, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e = binding.prologue_bwd(*args)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n in a:
        for other in (b, c, e):
            assert torch.equal(a[n], other[n]), n
