"""What the front end of the operators around the mixer refuses before anything
runs on the GPU, and calls that overlap."""
import pytest
import torch

from gated_delta_rule_93_b200 import GdrError, binding

pytestmark = pytest.mark.gpu


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def i32(*shape):
    return z(*shape, dtype=torch.int32)


def step(**kw):
    a = dict(q=z(5, 2, 64), k=z(5, 2, 64), v=z(5, 4, 32), g=z(5, 4), beta=z(5, 4),
             pool=z(6, 4, 32, 64), src=torch.arange(5, dtype=torch.int32, device="cuda"))
    return binding.step_slots(**dict(a, **kw))


def test_step_slots(cuda_device):
    step()
    bf16 = torch.bfloat16
    for error, kw in (
            (TypeError, dict(k=z(5, 2, 64, dtype=bf16))), (TypeError, dict(g=z(5, 4, dtype=bf16))),
            (TypeError, dict(q=z(5, 2, 64, dtype=torch.float16))), (TypeError, dict(src=z(5))),
            (TypeError, dict(pool=z(6, 4, 32, 64, dtype=bf16))), (TypeError, dict(q=None)),
            (TypeError, dict(stream=0)), (TypeError, dict(dst=i32(5).long())),
            (ValueError, dict(k=z(5, 1, 64))), (ValueError, dict(v=z(4, 4, 32))),
            (ValueError, dict(g=z(5, 4, 32))), (ValueError, dict(beta=z(5, 2))),
            (ValueError, dict(pool=z(6, 4, 64, 32))), (ValueError, dict(src=i32(4))),
            (ValueError, dict(src=i32(5, 1))), (ValueError, dict(dst=i32(4))),
            (ValueError, dict(cu_seqlens=i32(5))), (ValueError, dict(gate_scale=z(2))),
            (ValueError, dict(o=z(5, 4, 64))), (ValueError, dict(o=z(5, 32, 4).transpose(1, 2))),
            (ValueError, dict(q=z(5, 64, 2).transpose(1, 2))), (ValueError, dict(beta=z(4, 5).t())),
            (ValueError, dict(pool=z(6, 4, 64, 32).transpose(2, 3))),
            (ValueError, dict(pool=z(1, 4, 32, 64).expand(6, 4, 32, 64))),
            (ValueError, dict(beta=torch.zeros(5, 4))), (ValueError, dict(q=z(5, 128))),
            (GdrError, dict(q=z(5, 3, 64), k=z(5, 3, 64))),       # 4 value heads over 3 key heads
            (GdrError, dict(q=z(5 * 128 + 1)[1:].view(5, 2, 64))),  # 4 bytes off
            (GdrError, dict(v=z(5, 130)[:, :128].unflatten(1, (4, 32)))),  # rows 8 bytes off
            (GdrError, dict(q=z(5, 2, 48), k=z(5, 2, 48), pool=z(6, 4, 32, 48)))):
        with pytest.raises(error):
            step(**kw)


def test_slot_map(cuda_device):
    binding.slot_map(i32(3), i32(3), i32(3, 2), 4, 5)
    for error, a, kw in (
            (TypeError, (z(3), i32(3), i32(3, 2), 4, 5), {}),
            (TypeError, (i32(3), i32(3), i32(3, 2), 4.5, 5), {}),
            (ValueError, (i32(3), i32(2), i32(3, 2), 4, 5), {}),
            (ValueError, (i32(3), i32(3), i32(3), 4, 5), {}),
            (ValueError, (i32(3), i32(3), i32(2, 3).t(), 4, 5), {}),
            (ValueError, (i32(3), i32(3), i32(3, 2), -1, 5), {}),
            (ValueError, (i32(3), i32(3), i32(3, 2), 4, 2**31), {}),
            (ValueError, (i32(3), i32(3).cpu(), i32(3, 2), 4, 5), {}),
            (KeyError, (i32(3), i32(3), i32(3, 2), 4, 5), dict(out={"src": i32(3)})),
            (TypeError, (i32(3), i32(3), i32(3, 2), 4, 5), dict(out=[])),
            (GdrError, (i32(3), i32(3), i32(3, 0), 4, 5), {}),
            (GdrError, (i32(65537), i32(65537), i32(65537, 1), 4, 5), {})):
        with pytest.raises(error):
            binding.slot_map(*a, **kw)


def test_group_norm(cuda_device):
    x, w = z(5, 4, 64), z(64)
    binding.group_norm_fwd(x, x, w, w)
    for error, a, kw in (
            (TypeError, (x, x.bfloat16()), {}), (TypeError, (x.half(),), {}),
            (TypeError, (x, None, w.bfloat16()), {}), (TypeError, (x,), dict(eps="1")),
            (ValueError, (x, z(5, 4, 32)), {}), (ValueError, (x, None, z(4)), {}),
            (ValueError, (x, None, w, z(4, 64)), {}), (ValueError, (z(64),), {}),
            (ValueError, (x,), dict(y=z(5, 4, 128)[..., :64])),
            (ValueError, (z(5, 64, 4).transpose(1, 2),), {}),
            (GdrError, (x,), dict(eps=0.0)), (GdrError, (z(5, 1, 2048),), {}),
            (GdrError, (z(5, 0, 64),), {})):
        with pytest.raises(error):
            binding.group_norm_fwd(*a, **kw)
    for error, a, kw in (
            (ValueError, (z(5, 4, 128)[..., :64], x), {}), (TypeError, (x.bfloat16(), x), {}),
            (KeyError, (x, x), dict(out={})), (GdrError, (x, x, None, w), dict(workspace=z(1))),
            (ValueError, (x, x, None, w), dict(workspace=torch.zeros(1 << 20))),
            (TypeError, (x, x, None, w), dict(workspace=1 << 20))):
        with pytest.raises(error):
            binding.group_norm_bwd(*a, **kw)


def test_prologue(cuda_device):
    q, a, s = z(5, 2, 64), z(5, 4), z(4)
    binding.prologue_fwd(q, q, a, a, s)
    for error, args, kw in (
            (TypeError, (q, q.bfloat16(), a, a, s), {}), (ValueError, (q, q, a, z(5), s), {}),
            (ValueError, (q, q, z(5, 2), a, s), {}), (ValueError, (q, q, z(5, 4, 32), a, s), {}),
            (ValueError, (q, q, a, a, z(2)), {}), (TypeError, (q, q, a, a, s), dict(out=(q, q))),
            (ValueError, (q, q, a, a, s), dict(out=(q, q, a, a))),
            (GdrError, (z(5, 3, 64), z(5, 3, 64), a, a, s), {}),
            (GdrError, (z(5, 2, 48), z(5, 2, 48), a, a, s), {})):
        with pytest.raises(error):
            binding.prologue_fwd(*args, **kw)
    up = z(5, 4, 64)
    binding.prologue_bwd(q, q, a, a, s, up, up, a, a)
    for error, grads, kw in (
            (ValueError, (q, up, a, a), {}), (TypeError, (up.bfloat16(), up, a, a), {}),
            (ValueError, (up, up, up, a), {}), (GdrError, (up, up, a, a), dict(workspace=z(1))),
            (KeyError, (up, up, a, a), dict(out={}))):
        with pytest.raises(error):
            binding.prologue_bwd(q, q, a, a, s, *grads, **kw)
    torch.cuda.synchronize()


def test_two_calls_at_once(cuda_device):
    """The same gradient twice, each on its own stream with memory of its own, over and
    over: no call sees the other's partial sums."""
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    d = [(n(4000, 4, 128), n(4000, 4, 128), n(4000, 4, 128), n(128)) for _ in range(2)]
    want = [binding.group_norm_bwd(*x) for x in d]
    p = [(n(4000, 2, 64), n(4000, 2, 64), n(4000, 4), n(4000, 4), n(4).abs(), n(4000, 4, 64),
          n(4000, 4, 64), n(4000, 4), n(4000, 4)) for _ in range(2)]
    want_p = [binding.prologue_bwd(*x) for x in p]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((binding.group_norm_bwd(*d[i]), binding.prologue_bwd(*p[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in got[i]:
            assert all(torch.equal(a[k], want[i][k]) for k in ("dx", "dz", "dweight"))
            assert all(torch.equal(b[k], want_p[i][k]) for k in b)


def test_outputs_are_kept_for_the_stream_of_the_call(cuda_device):
    """With stream=, what the call allocates is not handed out again before that stream has
    used it, although nobody holds it any more."""
    x = torch.randn(20000, 16, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = binding.group_norm_bwd(x, x, x, w)["dweight"].clone()
    torch.cuda.synchronize()
    for _ in range(10):
        out = binding.group_norm_bwd(x, x, x, w, stream=side)
        dw = out["dweight"]
        del out  # its workspace and dx are free again on the current stream
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(8)]
        side.synchronize()
        assert torch.equal(dw, want)
        del junk
