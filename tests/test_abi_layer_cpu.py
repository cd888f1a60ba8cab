"""Refusals of the operators around the mixer: host-side checks, no GPU."""
import ctypes

import pytest
import torch

from gated_delta_rule_93_b200 import binding
from gated_delta_rule_93_b200.build import build

INVALID, UNSUPPORTED, WORKSPACE, OK = (binding.GDR_ERR_INVALID_ARG, binding.GDR_ERR_UNSUPPORTED,
                                       binding.GDR_ERR_WORKSPACE, binding.GDR_OK)


@pytest.fixture(scope="module")
def L():
    build()
    return binding.lib()


def ptr(off=0):
    return ctypes.c_void_p(0x10000 + off)


def caller(fn, order, defaults):
    def call(**kw):
        assert set(kw) <= set(defaults), kw
        a = dict(defaults, **kw)
        return fn(*(a[n] for n in order.split()))
    return call


def test_new_status_code(L):
    assert binding.status_string(binding.GDR_ERR_SLOT) == "GDR_ERR_SLOT"


def test_step_slots(L):
    p = ptr()
    order = ("q k v dt qs ks vs g gate beta gs norm pool slots ss src dst cu o R total Hk H dk dv "
             "stream")
    call = caller(L.gdr_step_slots, order, dict(
        q=p, k=p, v=p, dt=1, qs=256, ks=256, vs=512, g=p, gate=0, beta=p, gs=None, norm=0, pool=p,
        slots=9, ss=4 * 128 * 128, src=p, dst=None, cu=p, o=p, R=3, total=7, Hk=2, H=4, dk=128,
        dv=128, stream=None))
    for kw in (dict(dt=2), dict(gate=2), dict(norm=4), dict(norm=-1), dict(R=-1), dict(total=-1),
               dict(slots=-1), dict(Hk=3), dict(Hk=0), dict(q=None), dict(o=None), dict(src=None),
               dict(pool=None), dict(beta=None), dict(q=ptr(8)), dict(o=ptr(4)), dict(pool=ptr(4)),
               dict(src=ptr(2)), dict(dst=ptr(1)), dict(cu=ptr(3)), dict(qs=255), dict(qs=260),
               dict(vs=511), dict(ss=4 * 128 * 128 - 4), dict(ss=4 * 128 * 128 + 2),
               dict(cu=None), dict(vs=1 << 60), dict(R=1 << 30, total=1 << 30)):
        assert call(**kw) == INVALID, kw
        assert L.gdr_last_error_message()
    for kw in (dict(dk=100), dict(dv=256), dict(dk=0)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(R=0), dict(H=0), dict(total=0)):
        assert call(**kw) == OK, kw


def test_slot_map(L):
    p = ptr()
    call = caller(L.gdr_slot_map, "lens kept table ts R W slots max keep cu request src dst stream",
                  dict(lens=p, kept=p, table=p, ts=4, R=3, W=4, slots=9, max=12, keep=1, cu=p,
                       request=p, src=p, dst=p, stream=None))
    for kw in (dict(R=-1), dict(W=0), dict(slots=-1), dict(max=-1), dict(keep=2), dict(ts=3),
               dict(lens=None), dict(table=None), dict(cu=None), dict(dst=None), dict(src=None),
               dict(kept=ptr(2)), dict(cu=ptr(1))):
        assert call(**kw) == INVALID, kw
    assert call(R=65537) == UNSUPPORTED


def test_group_norm(L):
    p = ptr()
    fwd = caller(L.gdr_group_norm_fwd, "x z dt xs zs w b pc act center eps y rows G D stream",
                 dict(x=p, z=p, dt=1, xs=512, zs=512, w=p, b=p, pc=0, act=1, center=0, eps=1e-5, y=p,
                      rows=10, G=4, D=128, stream=None))
    need = L.gdr_group_norm_bwd_workspace_bytes(10, 4, 128, 1, 0)
    assert need > 0 and L.gdr_group_norm_bwd_workspace_bytes(10, 4, 2048, 1, 0) == 0
    bwd = caller(L.gdr_group_norm_bwd,
                 "dy x z dt xs zs w b pc act center eps dx dz dw db rows G D ws wsb stream",
                 dict(dy=p, x=p, z=p, dt=1, xs=512, zs=512, w=p, b=p, pc=0, act=1, center=0, eps=1e-5,
                      dx=p, dz=p, dw=p, db=p, rows=10, G=4, D=128, ws=p, wsb=need, stream=None))
    for call in (fwd, bwd):
        for kw in (dict(rows=-1), dict(G=0), dict(D=0), dict(dt=3), dict(act=3), dict(act=-1),
                   dict(pc=2), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(eps=float("inf")), dict(x=None), dict(x=ptr(1)), dict(z=ptr(1)),
                   dict(w=ptr(2)), dict(xs=511), dict(zs=100), dict(rows=1 << 50)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(D=1025), dict(G=1000), dict(D=1024, G=65)):
            assert call(**kw) == UNSUPPORTED, kw
    assert fwd(y=None) == INVALID and fwd(y=ptr(1)) == INVALID and fwd(rows=0) == OK
    for kw in (dict(z=None), dict(dy=None), dict(dx=None), dict(dx=ptr(2)), dict(dz=ptr(1)),
               dict(dw=ptr(2)), dict(ws=ptr(4))):
        assert bwd(**kw) == INVALID, kw
    assert bwd(ws=None) == WORKSPACE and bwd(wsb=need - 1) == WORKSPACE
    assert bwd(rows=0, dw=None, db=None, ws=None, wsb=0) == OK


def test_prologue(L):
    p = ptr()
    shape = dict(q=p, k=p, dt=1, qs=256, ks=256, a=p, gate=0, b=p, gs=p, norm=3, tokens=10, Hk=2, H=4,
                 dk=128, stream=None)
    fwd = caller(L.gdr_prologue_fwd, "q k dt qs ks a gate b gs norm qn kn g beta tokens Hk H dk stream",
                 dict(shape, qn=p, kn=p, g=p, beta=p))
    need = L.gdr_prologue_bwd_workspace_bytes(10, 4, 128, 0)
    bwd = caller(L.gdr_prologue_bwd,
                 "q k dt qs ks a gate b gs norm dqn dkn dg dbeta dq dk_ da db ds tokens Hk H dk ws wsb "
                 "stream",
                 dict(shape, dqn=p, dkn=p, dg=p, dbeta=p, dq=p, dk_=p, da=p, db=p, ds=p, ws=p, wsb=need))
    for call in (fwd, bwd):
        for kw in (dict(dt=2), dict(gate=5), dict(norm=4), dict(tokens=-1), dict(Hk=0), dict(H=0),
                   dict(Hk=3), dict(q=None), dict(a=None), dict(gs=None), dict(k=ptr(8)),
                   dict(b=ptr(4)), dict(qs=250), dict(ks=257), dict(tokens=1 << 50)):
            assert call(**kw) == INVALID, kw
        for kw in (dict(dk=96), dict(dk=0), dict(H=1 << 18)):
            assert call(**kw) == UNSUPPORTED, kw
    assert fwd(qn=None) == INVALID and fwd(g=ptr(4)) == INVALID and fwd(tokens=0) == OK
    assert bwd(ds=None) == INVALID and bwd(dq=None) == INVALID and bwd(da=ptr(8)) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(wsb=need - 4) == WORKSPACE


def test_cpu_tensors_are_refused(L):
    x, f = torch.zeros(4, 2, 64), torch.zeros(4, 2)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: binding.step_slots(x, x, x, f, f, torch.zeros(4, 2, 64, 64), i),
                 lambda: binding.slot_map(i, i, i[:, None], 4, 4),
                 lambda: binding.group_norm_fwd(x),
                 lambda: binding.group_norm_bwd(x, x),
                 lambda: binding.prologue_fwd(x, x, f, f, torch.ones(2)),
                 lambda: binding.prologue_bwd(x, x, f, f, torch.ones(2), x, x, f, f)):
        with pytest.raises(ValueError, match="CUDA"):
            call()



@pytest.mark.parametrize("stride,shape,row", [
    ((512, 64, 1), (5, 8, 64), 512), ((800, 64, 1), (5, 8, 64), 800),
    ((4800, 800, 64, 1), (3, 6, 8, 64), 800), ((64, 64, 1), (1, 8, 64), 512),
    ((9999, 800, 64, 1), (1, 6, 8, 64), 800), ((300, 7, 1), (5, 1, 64), 300)])
def test_rows_apart(L, stride, shape, row):
    assert binding.native().rows_apart(torch.zeros(60000).as_strided(shape, stride), "t") == row


@pytest.mark.parametrize("stride,shape", [
    ((512, 65, 1), (5, 8, 64)), ((1024, 128, 2), (5, 8, 64)), ((5000, 800, 64, 1), (3, 6, 8, 64)),
    ((0, 64, 1), (5, 8, 64)), ((64, 512, 1), (8, 5, 64)), ((100, 64, 1), (5, 8, 64))])
def test_rows_apart_refuses(L, stride, shape):
    with pytest.raises(ValueError, match="rows one distance apart"):
        binding.native().rows_apart(torch.zeros(60000).as_strided(shape, stride), "t")


def test_front_end_refuses_what_is_not_a_tensor(L):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(TypeError, match="x must be a torch.Tensor"):
        binding.group_norm_fwd([1.0])
    with pytest.raises(ValueError, match="act must be one of"):
        binding.group_norm_fwd(x, act="gelu")
    with pytest.raises(ValueError, match="act must be one of"):
        binding.group_norm_fwd(x, act=[])
    with pytest.raises(TypeError, match="expected 9 arguments"):
        binding.native().group_norm_fwd(x)
