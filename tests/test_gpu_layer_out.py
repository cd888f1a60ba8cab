"""``out`` of the operators around the mixer: dicts whose entries are in part None."""
import pytest
import torch

from gated_delta_rule_93_b200 import binding

pytestmark = pytest.mark.gpu


def n(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(sum(shape))).cuda()


def equal(got, want):
    return all(got[k] is w if got[k] is None or w is None else torch.equal(got[k], w)
               for k, w in want.items())


def test_norm_gradients_of_a_call_without_gate_and_bias_reused(cuda_device):
    """The dict of a call without z, weight and bias, whose entries for them are None, given
    to a call with all three: it gets what that call computes, its dx in the memory it had."""
    x, z, dy, w, b = n(9, 4, 64), n(9, 4, 64) + 1, n(9, 4, 64) - 1, n(64), n(64) + 2
    out = binding.group_norm_bwd(dy, x)
    assert [k for k, t in out.items() if t is None] == ["dz", "dweight", "dbias"]
    dx = out["dx"]
    got = binding.group_norm_bwd(dy, x, z, w, b, out=out)
    want = binding.group_norm_bwd(dy, x, z, w, b)
    torch.cuda.synchronize()
    assert got is out and got["dx"] is dx and equal(got, want)
    assert all(t is not None for t in got.values())
    # and again into the same tensors
    kept = dict(got)
    again = binding.group_norm_bwd(2 * dy, x, z, w, b, out=out)
    want = binding.group_norm_bwd(2 * dy, x, z, w, b)
    torch.cuda.synchronize()
    assert all(again[k] is kept[k] for k in kept) and equal(again, want)


def test_entries_without_an_input_stay(cuda_device):
    """Tensors of `out` for inputs that the call does not have are not touched."""
    x, dy = n(9, 4, 64), n(9, 4, 64) - 1
    out = dict(dx=torch.empty_like(x), dz=x.clone(), dweight=None, dbias=n(64))
    bias, dz = out["dbias"], out["dz"]
    got = binding.group_norm_bwd(dy, x, out=out)
    torch.cuda.synchronize()
    assert got["dbias"] is bias and got["dz"] is dz and got["dweight"] is None
    assert torch.equal(dz, x) and torch.equal(bias, n(64))
    assert torch.equal(got["dx"], binding.group_norm_bwd(dy, x)["dx"])


@pytest.mark.parametrize("none", [("dq",), ("dk", "da"), ("dq", "dk", "da", "db", "dgate_scale")])
def test_prologue_gradients(cuda_device, none):
    q, k, a, b, s = n(7, 2, 64), n(7, 2, 64) + 1, n(7, 4), n(7, 4) + 1, n(4).abs()
    up = n(7, 4, 64), n(7, 4, 64) - 1, n(7, 4) - 1, n(7, 4) + 2
    want = binding.prologue_bwd(q, k, a, b, s, *up)
    out = {name: None if name in none else torch.full_like(t, 7.0) for name, t in want.items()}
    got = binding.prologue_bwd(q, k, a, b, s, *up, out=out)
    torch.cuda.synchronize()
    assert got is out and equal(got, want)


def test_slot_map(cuda_device):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    args = i32([2, 0, 1]), i32([1, 0, 0]), i32([[0, 1], [2, 3], [4, 5]]), 6, 5
    want = binding.slot_map(*args)
    for none in want:
        out = {k: None if k == none else torch.full_like(t, 99) for k, t in want.items()}
        got = binding.slot_map(*args, out=out)
        torch.cuda.synchronize()
        assert got is out and equal(got, want)


def test_prologue_tuple(cuda_device):
    q, a, s = n(7, 2, 64), n(7, 4), n(4).abs()
    want = binding.prologue_fwd(q, q, a, a, s)
    g = torch.empty_like(a)
    got = binding.prologue_fwd(q, q, a, a, s, out=(None, None, g, None))
    torch.cuda.synchronize()
    assert got[2] is g and all(torch.equal(x, w) for x, w in zip(got, want))
