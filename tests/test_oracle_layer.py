"""Pins of the fp64 oracle of the operators around the mixer (CPU)."""
import numpy as np
import pytest

import oracle
from oracle import layer
from oracle.prologue import log_decay, prologue, sigmoid


def _rng(seed):
    return np.random.default_rng(seed)


def _differences(f, x, eps=1e-6):
    """Central differences of the scalar f by every entry of x."""
    out = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + eps
        up = f()
        x[i] = keep - eps
        out[i] = (up - f()) / (2 * eps)
        x[i] = keep
    return out


@pytest.mark.parametrize("gate", ["scalar", "channel"])
def test_step_slots_is_the_recurrence(gate):
    """Two requests from two slots equal the fp64 forward over each of them."""
    r = _rng(1)
    H, dk, dv, lens = 2, 4, 3, (3, 2)
    q, k = (r.standard_normal((5, H, dk)).astype(np.float32) for _ in range(2))
    v = r.standard_normal((5, H, dv)).astype(np.float32)
    g = -0.2 * r.random((5, H, dk) if gate == "channel" else (5, H)).astype(np.float32)
    beta = r.random((5, H)).astype(np.float32)
    pool = r.standard_normal((4, H, dv, dk))
    up = [x.astype(np.float64) for x in (q, k, v, g, beta)]
    o, after = layer.step_slots(*up, pool, [2, 0], dst=[-1, -1, 1, 0, -1], cu=[0, 3, 5])
    at = 0
    for n, slot, kept in zip(lens, (2, 0), ({2: 1}, {0: 0})):
        part = [x[None, at:at + n] for x in (q, k, v, g, beta)]
        ro, rS = oracle.gdr_fwd(*part, pool[None, slot], gate=gate)
        np.testing.assert_allclose(o[at:at + n], ro[0], atol=1e-12)
        if 2 in kept:
            np.testing.assert_allclose(after[1], rS[0], atol=1e-12)
        at += n
    # slot 0 keeps the state after the second request's first token only
    _, one = oracle.gdr_fwd(*[x[None, 3:4] for x in (q, k, v, g, beta)], pool[None, 0], gate=gate)
    np.testing.assert_allclose(after[0], one[0], atol=1e-12)
    np.testing.assert_array_equal(after[2:], pool[2:])


def test_step_slots_shares_key_heads_and_maps_raw_projections():
    r = _rng(2)
    q, k = r.standard_normal((2, 2, 4)), r.standard_normal((2, 2, 4))
    v, a, b = r.standard_normal((2, 4, 3)), r.standard_normal((2, 4)), r.standard_normal((2, 4))
    s = np.array([0.1, 0.2, 0.3, 0.4])
    pool = r.standard_normal((3, 4, 3, 4))
    o, after = layer.step_slots(q, k, v, a, b, pool, [1, -1], gate_scale=s, norm_q=True,
                                norm_k=True)
    unit = lambda x: np.repeat(x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6), 2, axis=1)
    o2, after2 = layer.step_slots(unit(q), unit(k), v, log_decay(a[None], s)[0], sigmoid(b), pool,
                                  [1, -1])
    np.testing.assert_allclose(o, o2, atol=1e-13)
    np.testing.assert_allclose(after, after2, atol=1e-13)
    np.testing.assert_array_equal(after[[0, 2]], pool[[0, 2]])  # a new request's state is dropped


def test_slot_map_by_hand():
    table = np.array([[4, 5], [0, 1], [2, 3], [6, 7]])
    cu, src, request, dst, bad = layer.slot_map([2, 0, 1, 1], [1, 2, 2, 0], table, 8, 6, True)
    assert cu.tolist() == [0, 2, 2, 3, 4] and src.tolist() == [4, -2, 3, -1] and not bad
    assert request.tolist() == [0, 0, 2, 3, -1, -1] and dst.tolist() == [4, 5, 2, 6, -1, -1]
    cu, src, request, dst, bad = layer.slot_map([3, 0, 1, 1], [1, 2, 2, 0], table, 8, 6, False)
    assert cu.tolist() == [0, 3, 3, 4, 5] and dst.tolist() == [-1, -1, 4, 2, 6, -1] and not bad
    assert layer.slot_map([3, 0, 1, 1], [1, 2, 2, 0], table, 8, 6, True)[1].tolist() == [-2, -2, 3, -1]


@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("act", ["silu", "sigmoid", "none"])
@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("channel", [True, False])
def test_group_norm_gradient_against_differences(gated, act, center, channel):
    r = _rng(3)
    x, dy = r.standard_normal((2, 2, 3)), r.standard_normal((2, 2, 3))
    z = r.standard_normal((2, 2, 3)) if gated else None
    w, b = (r.standard_normal((2, 3) if channel else (3,)) for _ in range(2))
    f = lambda: float((dy * layer.group_norm(x, z, w, b, act, center)).sum())
    got = layer.group_norm_grad(dy, x, z, w, b, act, center)
    for name, wrt in (("dx", x), ("dz", z), ("dweight", w), ("dbias", b)):
        if wrt is not None:
            np.testing.assert_allclose(got[name], _differences(f, wrt), atol=1e-7)


def test_group_norm_statistics():
    r = _rng(4)
    x = 3 + r.standard_normal((5, 2, 16))
    y = layer.group_norm(x, act="none", center=True)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-13)
    np.testing.assert_allclose((y * y).mean(-1), 1, atol=1e-4)
    np.testing.assert_allclose((layer.group_norm(x, act="none") ** 2).mean(-1), 1, atol=1e-4)
    # a group's scale does not matter, its neighbours neither
    big = x.copy()
    big[:, 1] *= 1000
    np.testing.assert_allclose(layer.group_norm(big, act="none"), layer.group_norm(x, act="none"),
                               atol=1e-5)


@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("norm_q,norm_k", [(True, True), (False, True), (True, False)])
def test_prologue_gradient_against_differences(gate, norm_q, norm_k):
    r = _rng(5)
    t, Hk, H, d = 2, 2, 4, 3
    q, k = r.standard_normal((t, Hk, d)), r.standard_normal((t, Hk, d))
    a = r.standard_normal((t, H, d) if gate == "channel" else (t, H))
    b, s = r.standard_normal((t, H)), 0.1 + r.random(H)
    ups = [r.standard_normal((t, H, d)), r.standard_normal((t, H, d)), r.standard_normal(a.shape),
           r.standard_normal(b.shape)]

    def f():
        qn, kn, _, beta = prologue(q, k, a[None], b, s, norm_q, norm_k)
        outs = (np.repeat(qn, H // Hk, 1), np.repeat(kn, H // Hk, 1), log_decay(a[None], s)[0], beta)
        return float(sum((u * o).sum() for u, o in zip(ups, outs)))

    got = layer.prologue_grad(q, k, a, b, s, *ups, norm_q=norm_q, norm_k=norm_k)
    for name, wrt in (("dq", q), ("dk", k), ("da", a), ("db", b), ("dgate_scale", s)):
        np.testing.assert_allclose(got[name], _differences(f, wrt), atol=1e-7)
