"""GPU parity of gdr_group_norm_fwd / _bwd against the fp64 oracle.

Tolerances (max|d| / max|ref|).  The longest chain of fp32 roundings behind an
output: up to 32 elements of a lane in sequence and 5 lane steps for the mean,
as many for the mean square, and in the backward as many for its two means,
plus about 20 for exp, reciprocal, rsqrt and the products: 4 * 37 + 20 < 256,
so 256 * 2^-24 = 1.6e-5 of the largest terms.  An output's largest terms
exceed its largest value by at most the factor `amp` = 4 that centring and
dx's cancellation (h - mean h - n mean h n) take at these inputs.  Sums over
rows: 2^-24 per addition in sequence (rows / rows in flight + 64), relative to the
sum of the terms' sizes, which the test measures.  bf16 outputs are rounded
once more, by at most 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import binding
from oracle import layer

pytestmark = pytest.mark.gpu

FP32 = 4 * 256 * 2.0**-24
BF16 = 2.0**-8


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(rows, G, D, dtype, gated=True, affine="group", bias=True, apart=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)

    def strided(scale):
        t = (n(rows, G * D + apart) * scale).to(dtype).cuda()
        return t[:, : G * D].unflatten(1, (G, D)) if apart else t.view(rows, G, D)

    shape = (G, D) if affine == "channel" else (D,)
    return dict(x=strided(0.7), z=strided(1.5) if gated else None,
                weight=None if affine == "none" else (1 + 0.3 * n(*shape)).cuda(),
                bias=(0.3 * n(*shape)).cuda() if bias else None,
                dy=n(rows, G, D).to(dtype).cuda())


def close(got, want, tol, what, scale=None):
    got = f64(got)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    if got.size:
        e = np.abs(got - want).max() / (np.abs(want).max() if scale is None else scale)
        assert e <= tol, f"{what}: {e:.3e} > {tol:.3e}"


def check(d, act, center, dtype, eps=1e-5, **kw):
    names = ("x", "z", "weight", "bias")
    args = [d[n] for n in names]
    up = [f64(a) for a in args]
    y = binding.group_norm_fwd(*args, act=act, center=center, eps=eps, **kw)
    got = binding.group_norm_bwd(d["dy"], *args, act=act, center=center, eps=eps, **kw)
    torch.cuda.synchronize()
    low = BF16 if dtype == torch.bfloat16 else 0.0
    assert y.dtype == dtype and got["dx"].dtype == torch.float32
    close(y, layer.group_norm(*up, act, center, eps), FP32 + low, "y")
    want = layer.group_norm_grad(f64(d["dy"]), *up, act, center, eps)
    close(got["dx"], want["dx"], FP32, "dx")
    if d["z"] is None:
        assert got["dz"] is None
    else:
        assert got["dz"].dtype == dtype
        close(got["dz"], want["dz"], FP32 + low, "dz")
    # |terms| of the sums over rows, from the formula with every sign made equal
    rows = d["x"].shape[0]
    n, _, lin = layer._normalised(up[0], up[2], up[3], center, eps)
    f, df = layer._act(act, lin if up[1] is None else up[1])
    dl = np.abs(f64(d["dy"]) * (df if up[1] is None else f))
    for name, p, term in (("dweight", d["weight"], dl * np.abs(n)), ("dbias", d["bias"], dl)):
        if p is None:
            assert got[name] is None
            continue
        size = term.sum((0, 1) if p.dim() == 1 else 0).max() if rows else 1.0
        close(got[name], want[name], FP32 + (rows / 100 + 64) * 2.0**-24, name, scale=size)
    return y, got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act,gated", [("silu", True), ("sigmoid", True), ("silu", False),
                                       ("sigmoid", False), ("none", False), ("none", True)])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("affine", ["group", "channel", "none"])
def test_forms(cuda_device, dtype, act, gated, center, affine):
    d = make(37, 5, 128, dtype, gated, affine, bias=affine != "none", seed=1)
    check(d, act, center, dtype)


# one element, below and above a vector, odd, every number of vectors a lane holds, the widest
@pytest.mark.parametrize("D", [1, 2, 7, 8, 20, 31, 32, 33, 48, 63, 64, 80, 95, 96, 100, 127, 191, 192,
                               250, 252, 255, 256, 257, 500, 512, 513, 1000, 1020, 1023, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("affine", ["group", "channel"])
def test_widths(cuda_device, D, dtype, affine):
    d = make(19, 3, D, dtype, True, affine, seed=D)
    # (one element: n is +-1, and dx cancels to nothing but rounding next to it)
    if D == 1:
        d["x"].abs_().add_(0.5)
    check(d, "silu", D > 2, dtype) if D > 2 else check(d, "silu", False, dtype, eps=0.5)


@pytest.mark.parametrize("rows,G", [(1, 1), (1, 16), (2, 1000), (3000, 1), (4097, 5), (700, 31),
                                    (9001, 16)])
@pytest.mark.parametrize("affine", ["group", "channel"])
def test_rows_and_groups(cuda_device, rows, G, affine):
    d = make(rows, G, 64, torch.bfloat16, True, affine, seed=rows)
    check(d, "silu", False, torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("apart", [8, 128, 5])
def test_rows_apart(cuda_device, dtype, apart):
    """Slices of a fused projection; 5 elements apart breaks every alignment."""
    check(make(50, 4, 128, dtype, True, "group", apart=apart, seed=apart), "silu", False, dtype)


def test_tokens_in_two_dimensions(cuda_device):
    d = make(24, 4, 64, torch.bfloat16, True, "group", bias=False, apart=64, seed=6)
    four = lambda t: t.unflatten(0, (4, 6))
    y = binding.group_norm_fwd(four(d["x"]), four(d["z"]), d["weight"])
    got = binding.group_norm_bwd(four(d["dy"]), four(d["x"]), four(d["z"]), d["weight"])
    y1 = binding.group_norm_fwd(d["x"], d["z"], d["weight"])
    got1 = binding.group_norm_bwd(d["dy"], d["x"], d["z"], d["weight"])
    assert y.shape == (4, 6, 4, 64) and torch.equal(y.flatten(0, 1), y1)
    assert torch.equal(got["dx"].flatten(0, 1), got1["dx"])
    assert torch.equal(got["dweight"], got1["dweight"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("center", [True, False])
def test_rows_of_zeros_and_constants(cuda_device, dtype, center):
    """A zero row stays zero (or the bias) with finite gradients."""
    d = make(6, 2, 64, dtype, True, "group", seed=7)
    d["x"][1] = 0.0
    d["x"][3] = 2.0
    check(d, "silu", center, dtype, eps=1e-3)


def test_gates_far_out(cuda_device):
    """z at +-100 and +-80: the activation is 0 or z, nothing overflows."""
    d = make(8, 2, 64, torch.float32, True, "group", seed=8)
    for i, x in enumerate((100.0, -100.0, 80.0, -80.0, 0.0)):
        d["z"][i] = x
    check(d, "silu", False, torch.float32)
    check(d, "sigmoid", False, torch.float32)


def test_nan_stays_in_its_group(cuda_device):
    """A NaN or an infinity reaches its own group of its own token only."""
    d = make(40, 4, 96, torch.float32, True, "none", bias=False, seed=9)
    y0 = binding.group_norm_fwd(d["x"], d["z"])
    g0 = binding.group_norm_bwd(d["dy"], d["x"], d["z"])
    d["x"][11, 2, 5], d["x"][20, 0, 95] = float("nan"), float("inf")
    y1 = binding.group_norm_fwd(d["x"], d["z"])
    g1 = binding.group_norm_bwd(d["dy"], d["x"], d["z"])
    torch.cuda.synchronize()
    keep = torch.ones(40, 4, dtype=torch.bool, device="cuda")
    keep[11, 2] = keep[20, 0] = False
    for a, b in ((y0, y1), (g0["dx"], g1["dx"]), (g0["dz"], g1["dz"])):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(y1[11, 2]).all()


def test_in_place_and_no_rows(cuda_device):
    d = make(30, 4, 64, torch.bfloat16, True, "group", seed=10)
    y = binding.group_norm_fwd(d["x"], d["z"], d["weight"], d["bias"])
    x = d["x"].clone()
    assert binding.group_norm_fwd(x, d["z"], d["weight"], d["bias"], y=x) is x
    torch.cuda.synchronize()
    assert torch.equal(x, y)
    e = make(0, 4, 64, torch.bfloat16, True, "group", seed=10)
    assert binding.group_norm_fwd(e["x"], e["z"], e["weight"], e["bias"]).shape == (0, 4, 64)
    got = binding.group_norm_bwd(e["dy"], e["x"], e["z"], e["weight"], e["bias"])
    torch.cuda.synchronize()
    assert got["dx"].shape == (0, 4, 64) and not got["dweight"].any() and not got["dbias"].any()


def test_offsets_beyond_32_bits(cuda_device):
    """More than 2^31 elements behind the first row."""
    apart = 1 << 22
    rows = (1 << 31) // apart + 2
    buf = torch.empty(rows * apart, dtype=torch.bfloat16, device="cuda")
    x = buf.view(rows, apart)[:, :128].unflatten(1, (2, 64))
    d = make(rows, 2, 64, torch.bfloat16, True, "group", seed=11)
    x.copy_(d["x"])
    y = binding.group_norm_fwd(x, d["z"], d["weight"])
    got = binding.group_norm_bwd(d["dy"], x, d["z"], d["weight"])
    y1 = binding.group_norm_fwd(d["x"], d["z"], d["weight"])
    got1 = binding.group_norm_bwd(d["dy"], d["x"], d["z"], d["weight"])
    torch.cuda.synchronize()
    assert torch.equal(y, y1) and torch.equal(got["dx"], got1["dx"])


def test_gradient_against_differences(cuda_device):
    """The kernel's own forward, differenced (fp32, so a coarse bar: half a step of 1e-2
    leaves truncation 1e-4 and rounding 2^-24 / 1e-2 per term)."""
    d = make(3, 2, 32, torch.float32, True, "channel", seed=12)
    args = [d[n] for n in ("x", "z", "weight", "bias")]
    got = binding.group_norm_bwd(d["dy"], *args, center=True)
    loss = lambda: float((binding.group_norm_fwd(*args, center=True).double() * d["dy"].double()).sum())
    for name, t in zip(("dx", "dz", "dweight", "dbias"), args):
        for at in ((0,) * t.dim(), tuple(s - 1 for s in t.shape)):
            keep = float(t[at])
            t[at] = keep + 1e-2
            up = loss()
            t[at] = keep - 1e-2
            down = loss()
            t[at] = keep
            assert abs((up - down) / 2e-2 - float(got[name][at])) < 5e-3, (name, at)


def test_same_bits_other_stream_and_graph(cuda_device):
    """Twice the same call, on a side stream with its own workspace, and two captures that
    share one workspace, replayed one after the other: the same bits."""
    d = make(5000, 4, 128, torch.bfloat16, True, "group", seed=13)
    args = [d["dy"]] + [d[n] for n in ("x", "z", "weight", "bias")]
    a, b = binding.group_norm_bwd(*args), binding.group_norm_bwd(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = binding.group_norm_bwd(*args, stream=side)
    side.synchronize()
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.group_norm_bwd(*args, workspace=ws))
        graphs.append(g)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for name in a:
        for other in (b, c, *outs):
            assert torch.equal(a[name], other[name]), name
