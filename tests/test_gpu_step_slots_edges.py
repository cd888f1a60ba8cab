"""gdr_step_slots at the edges of its batches of prepared tokens and of its tensors:
what lies around them is NaN (and slots that nobody named), so that a read or a write
beyond them shows."""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import SLOT_ZERO, binding
from oracle import layer
from test_gpu_step_slots import call, close, expect, f64, i32, make, tolerance

pytestmark = pytest.mark.gpu

PAD = 64  # elements before and after, whole 16-byte units of every type


def framed(t, fill):
    """A copy of t in the middle of a buffer of `fill`, and the buffer."""
    whole = torch.full((t.numel() + 2 * PAD,), fill, dtype=t.dtype, device="cuda")
    inner = whole[PAD:PAD + t.numel()].view(t.shape)
    inner.copy_(t)
    return inner, whole


def frame(whole):
    return torch.cat([whole[:PAD], whole[-PAD:]])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("cu,runs", [
    ([-5, 3, 99, 2], [(0, 3), (3, 6), (6, 6)]),               # below 0, behind the end, falling
    ([-2**31, -7, 2, 2**31 - 1], [(0, 0), (0, 2), (2, 6)]),   # a request before all tokens
    ([7, 9, 12, 2**31 - 1], [(6, 6)] * 3),                    # all behind the end
    ([4, 4, 5, 4], [(4, 4), (4, 5), (5, 5)])])                # tokens of nobody on both sides
def test_offsets_are_clamped(cuda_device, dtype, gate, cu, runs):
    """Just the tokens of the clamped offsets run, from and to the slots they name."""
    d = make([2, 2, 2], 1, 2, 32, 32, dtype, gate, slots=12, seed=14)
    for n in ("q", "k", "v", "g", "beta"):
        d[n], _ = framed(d[n], float("nan"))
    pool, pool_whole = framed(d["pool"], 5.0)
    src, dst = i32([0, 1, 2]), framed(i32([3, 4, 5, 6, 7, 8]), 11)[0]
    o, o_whole = framed(torch.full_like(d["v"], 7.0), 9.0)
    # the oracle, a request at a time on the tokens that run
    want_o, want = f64(o), f64(pool)
    for r, (lo, hi) in enumerate(runs):
        part = [f64(d[n])[lo:hi] for n in ("q", "k", "v", "g", "beta")]
        ro, rp = layer.step_slots(*part, f64(pool), [r], list(range(3 + lo, 3 + hi)), [0, hi - lo])
        want_o[lo:hi] = ro
        want[3 + lo:3 + hi] = rp[3 + lo:3 + hi]
    binding.step_slots(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, src, dst=dst,
                       cu_seqlens=i32(cu), o=o)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    close(o, want_o, tolerance(32, 4, dtype), "o")
    close(pool, want, tolerance(32, 4), "pool")
    ran = sorted(t for lo, hi in runs for t in range(lo, hi))
    idle = [t for t in range(6) if t not in ran]
    assert (o[idle] == 7.0).all() and (frame(o_whole) == 9.0).all()
    same = [s for s in range(12) if s - 3 not in ran]
    assert np.array_equal(f64(pool)[same], want[same]) and (frame(pool_whole) == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["scalar", "channel"])
@pytest.mark.parametrize("tokens", [7, 8, 9, 16, 17])
@pytest.mark.parametrize("dv", [32, 128])
def test_lengths_around_the_eight_tokens_prepared_at_a_time(cuda_device, dtype, gate, tokens, dv):
    """A batch that is full, one short of it and one over, twice; beside it a request of one
    token and a new one of as many; the state kept after some tokens, the last among them."""
    lens = [tokens, 1, tokens]
    d = make(lens, 1, 2, 64, dv, dtype, gate, True, slots=12, seed=tokens)
    for n in ("q", "k", "v", "g", "beta"):
        d[n], _ = framed(d[n], float("nan"))
    kept = [-1] * sum(lens)
    kept[min(6, tokens - 1)], kept[tokens - 1], kept[tokens], kept[-1] = 2, 3, 4, 5
    src, dst = i32([0, 1, SLOT_ZERO]), i32(kept)
    ro, rp = expect(d, src, dst)
    o, o_whole = framed(torch.zeros_like(d["v"]), 9.0)
    call(d, src, dst, o=o)
    torch.cuda.synchronize()
    assert binding.device_status() == 0 and (frame(o_whole) == 9.0).all()
    close(o, ro, tolerance(64, tokens, dtype), "o")
    close(d["pool"], rp, tolerance(64, tokens), "pool")
    last = binding.step_slots(d["q"], d["k"], d["v"], d["g"], d["beta"], d["pool"], i32([3, 4, 5]),
                              cu_seqlens=d["cu"], gate_scale=d["scale"], norm_q=True, norm_k=True)
    assert torch.isfinite(last).all()
