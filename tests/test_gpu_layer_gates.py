"""The gates' softplus and sigmoid, element by element over the whole range of logits.

Bounds, relative, in units of 2^-23 (a rounding is half a unit; ex2.approx is documented with 2
units, rcp.approx with 1):
* e^-|x|: 2, and a half for the factor that makes up for the rounded exponent: 2.5.
* softplus = max(x, 0) + 2 s p(s^2), s = e / (2 + e): e 2.5, the sum 0.5, its reciprocal 1, s 0.5,
  the series 0.6 with its fit (4.5e-9), the last fma 0.5: below 6.
* sigmoid = (1 or e) / (1 + e): 2.5 + 0.5 + 1 + 0.5 = 4.5.
* every product behind them 0.5 more.
Below -87.3 (e^x under the smallest normal number) they are 0.
The activations of the output norm keep their argument's rounding: 4 + |x|, 0 below -87.3.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import SLOT_ZERO, binding

pytestmark = pytest.mark.gpu

U = 2.0**-23


def logits(n):
    """From -87 to 87, evenly, and close to zero from both sides; fp32 values in fp64."""
    near = np.logspace(-30, 0, n // 8)
    x = np.concatenate([np.linspace(-87, 87, n - 2 * (n // 8)), near, -near]).astype(np.float32)
    return x.astype(np.float64)


def dev(x):
    return torch.tensor(np.asarray(x, dtype=np.float32), device="cuda")


def f64(t):
    return t.double().cpu().numpy()


def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1 + e)


def slope(x):
    e = np.exp(-np.abs(x))
    return e / (1 + e) ** 2


def within(got, want, units, what):
    e = np.abs(f64(got).reshape(want.shape) - want) / np.abs(want) / U
    worst, at = float(e.max()), int(e.argmax())
    assert worst <= units, f"{what}: {worst:.2f} > {units} units (reference {want.flat[at]:.3e})"


@pytest.mark.parametrize("gate", ["scalar", "channel"])
def test_prologue(cuda_device, gate):
    tokens, H, d = 1 << 14, 4, 32
    b = logits(tokens * H).reshape(tokens, H)
    a = logits(tokens * H * d).reshape(tokens, H, d) if gate == "channel" else b
    q = torch.ones(tokens, 1, d, device="cuda")
    one = torch.ones(H, device="cuda")
    _, _, g, beta = binding.prologue_fwd(q, q, dev(a), dev(b), one)
    within(g, -softplus(a), 6.5, "g")
    within(beta, sigmoid(b), 4.5, "beta")
    up = torch.ones(tokens, H, d, device="cuda")
    ones = torch.ones_like(beta)
    got = binding.prologue_bwd(q, q, dev(a), dev(b), one, up, up, torch.ones_like(g), ones)
    within(got["da"], -sigmoid(a), 5.5, "da")


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("several", [False, True])
def test_step_slots(cuda_device, gate, several):
    """A state of ones under a zero key shows alpha = e^-softplus(a) (its exponent's error,
    |g| 6.5 units, and 2 of expf); an empty one under a unit key shows beta."""
    R, H, d = 2048, 4, 64
    cu = torch.arange(R + 1, dtype=torch.int32, device="cuda") if several else None
    a = logits(R * H).reshape(R, H)
    g = dev(a)[..., None].expand(R, H, d).contiguous() if gate == "channel" else dev(a)
    pool = torch.ones(R, H, 32, d, device="cuda")
    k, v = torch.zeros(R, 1, d, device="cuda"), torch.ones(R, H, 32, device="cuda")
    slots = torch.arange(R, dtype=torch.int32, device="cuda")
    one = torch.ones(H, device="cuda")
    binding.step_slots(k, k, v, g, dev(a), pool, slots, cu_seqlens=cu, gate_scale=one)
    sp = softplus(a)[..., None, None]
    e = np.abs(f64(pool) - np.exp(-sp)) / (np.exp(-sp) * (6.5 * sp + 2.5) * U + 2.0**-126)
    assert float(e.max()) <= 1
    k[..., 0] = 1
    binding.step_slots(k, k, v, g, dev(a), pool, torch.full_like(slots, SLOT_ZERO), dst=slots,
                       cu_seqlens=cu, gate_scale=one)
    within(pool[..., 0], np.repeat(sigmoid(a)[..., None], 32, axis=2), 5, "beta")
    assert not pool[..., 1:].any()


FAR = [-np.inf, -3e38, -1e4, -200.0, -104.0, -89.0, 89.0, 104.0, 200.0, 1e4, 3e38, np.inf, np.nan]


@pytest.mark.parametrize("gate", ["scalar", "channel"])
def test_far_logits(cuda_device, gate):
    """Beyond the range of e^x, at the infinities and at NaN: the limits."""
    d = 32
    x = dev(FAR)[:, None]
    a = x[..., None].expand(len(FAR), 1, d).contiguous() if gate == "channel" else x
    q = torch.ones(len(FAR), 1, d, device="cuda")
    one, up = torch.ones(1, device="cuda"), torch.ones(len(FAR), 1, d, device="cuda")
    _, _, g, beta = binding.prologue_fwd(q, q, a, x, one)
    got = binding.prologue_bwd(q, q, a, x, one, up, up, torch.ones_like(a), torch.ones_like(x))
    g, da = (f64(t).reshape(len(FAR), -1)[:, 0] for t in (g, got["da"]))
    beta, db = f64(beta)[:, 0], f64(got["db"])[:, 0]
    assert np.isnan([g[-1], da[-1], beta[-1], db[-1]]).all()
    X = np.asarray(FAR[:-1], dtype=np.float32)
    tiny = 2.0**-126
    assert (np.abs(g[:6]) <= tiny).all() and (np.abs(da[:6]) <= tiny).all()
    assert (beta[:6] <= tiny).all() and (np.abs(db[:-1]) <= tiny).all()
    assert (g[6:-1] == -X[6:]).all() and (da[6:-1] == -1).all() and (beta[6:-1] == 1).all()


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_norm_activations(cuda_device, act):
    """l = 1 (weights of zero, biases of one), so that y = act(z) and dz = dy act'(z)."""
    rows, D = 1 << 12, 128
    z = logits(rows * D).reshape(rows, 1, D)
    x = torch.ones(rows, 1, D, device="cuda")
    w, b = torch.zeros(D, device="cuda"), torch.ones(D, device="cuda")
    s = sigmoid(z)
    y = binding.group_norm_fwd(x, dev(z), w, b, act=act)
    want = z * s if act == "silu" else s
    e = np.abs(f64(y) - want) / (np.abs(want) * (5 + np.abs(z)) * U + 2.0**-126)
    assert float(e.max()) <= 1
    dz = binding.group_norm_bwd(x, x, dev(z), w, b, act=act)["dz"]
    # s is off by ds = (4 + |z|) s and t = 1 - s <= 1 by ds + 1/2.  The sigmoid's slope s t is
    # off by t ds + s dt <= ds + s (ds + 1/2), SiLU's s + (z s) t by ds + |z| (ds + s (ds + 1/2)),
    # and each of up to four more roundings by half a unit of terms no larger than (1 + |z|) s.
    ds, slopes = (4 + np.abs(z)) * s, slope(z)
    product = ds + s * (ds + 0.5)
    want, bound = (s + z * slopes, ds + np.abs(z) * product + 2 * (1 + np.abs(z)) * s) \
        if act == "silu" else (slopes, product + 2 * s)
    e = np.abs(f64(dz) - want) / (bound * U + 2.0**-126)
    assert float(e.max()) <= 1
