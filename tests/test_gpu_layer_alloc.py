"""How the operators around the mixer allocate: as torch.empty does, seen by what watches it."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gated_delta_rule_93_b200 import SLOT_SKIP, binding

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    """Counts the allocations that go through the dispatcher."""

    def __init__(self):
        super().__init__()
        self.sizes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.sizes.append(tuple(out.shape))
        return out


@pytest.fixture
def deterministic():
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def calls():
    n = lambda *s: torch.randn(*s, device="cuda")
    q, v, a, s = n(5, 2, 64), n(5, 4, 64), n(5, 4), n(4).abs()
    i = torch.arange(5, dtype=torch.int32, device="cuda")
    pool, up, w = n(5, 4, 64, 64), n(5, 4, 64), n(64)
    side = torch.cuda.Stream()
    return {
        "step": (lambda **k: binding.step_slots(q, q, v, a, a, pool, i, **k), [(5, 4, 64)]),
        "map": (lambda **k: binding.slot_map(i, i * 0, i[:, None], 5, 7, **k), [(25,)]),
        "norm": (lambda **k: binding.group_norm_fwd(v, **k), [(5, 4, 64)]),
        "norm gradient": (lambda **k: binding.group_norm_bwd(v, v, None, w, **k),
                          [(5, 4, 64), (64,)]),
        "prologue": (lambda **k: binding.prologue_fwd(q, q, a, a, s, **k),
                     [(5, 4, 64)] * 2 + [(5, 4)] * 2),
        "prologue gradient": (lambda **k: binding.prologue_bwd(q, q, a, a, s, up, up, a, a, **k),
                              [(5, 2, 64)] * 2 + [(5, 4)] * 2 + [(4,)]),
    }, side


@pytest.mark.parametrize("op", ["step", "map", "norm", "norm gradient", "prologue",
                                "prologue gradient"])
@pytest.mark.parametrize("other", [False, True])
def test_a_dispatch_mode_sees_the_outputs(cuda_device, op, other):
    run, side = calls()
    run, sizes = run[op]
    torch.cuda.synchronize()
    with Seen() as seen:
        run(**({"stream": side} if other else {}))
    torch.cuda.synchronize()
    assert seen.sizes[:len(sizes)] == sizes
    assert binding.device_status() in (0, binding.GDR_ERR_SLOT)


def test_new_memory_is_filled_where_that_is_asked_for(cuda_device, deterministic):
    """With deterministic algorithms torch fills new memory with NaN: rows of o that no
    request covers hold that, as after torch.empty."""
    n = lambda *s: torch.randn(*s, device="cuda")
    q, v, a = n(4, 2, 64), n(4, 4, 64), n(4, 4)
    src = torch.tensor([0, SLOT_SKIP, 1, 2], dtype=torch.int32, device="cuda")
    o = binding.step_slots(q, q, v, a, a.sigmoid(), n(4, 4, 64, 64), src)
    torch.cuda.synchronize()
    assert torch.isnan(o[1]).all() and torch.isfinite(o[[0, 2, 3]]).all()
