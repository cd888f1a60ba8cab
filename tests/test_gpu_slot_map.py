"""gdr_slot_map against plain loops: whole numbers, equal."""
import numpy as np
import pytest
import torch

from gated_delta_rule_93_b200 import binding
from oracle import layer

pytestmark = pytest.mark.gpu


def check(lens, kept, table, slots, max_tokens, keep_all, device_table=None, **kw):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    got = binding.slot_map(dev(lens), dev(kept), dev(table) if device_table is None else device_table,
                           slots, max_tokens, keep_all=keep_all, **kw)
    torch.cuda.synchronize()
    want = layer.slot_map(lens, kept, np.asarray(table), slots, max_tokens, keep_all)
    for name, w in zip(("cu_seqlens", "src", "request", "dst"), want):
        assert got[name].dtype == torch.int32
        np.testing.assert_array_equal(got[name].cpu().numpy(), w, err_msg=name)
    assert binding.device_status() == (binding.GDR_ERR_SLOT if want[4] else 0)
    return got


def batch(R, W, seed, longest=None):
    r = np.random.default_rng(seed)
    table = r.permutation(R * W + 5)[: R * W].reshape(R, W)
    return r.integers(0, (longest or W) + 1, R), r.integers(0, W + 1, R), table, R * W + 5


# around a block's 256 requests, and the most requests a call takes
@pytest.mark.parametrize("R", [1, 2, 31, 255, 256, 257, 700, 4096, 65536])
@pytest.mark.parametrize("keep_all", [True, False])
def test_random_batches(cuda_device, R, keep_all):
    W = 1 + R % 7
    lens, kept, table, slots = batch(R, W, seed=R)
    check(lens, kept, table, slots, int(lens.sum()) + R % 300, keep_all)


def test_long_requests(cuda_device):
    """Prefill lengths: only the last state is kept."""
    lens, kept, table, slots = batch(40, 2, seed=3, longest=3000)
    check(lens, kept, table, slots, int(lens.sum()), False)


@pytest.mark.parametrize("keep_all", [True, False])
def test_no_tokens_and_no_requests(cuda_device, keep_all):
    check([0, 0, 0], [1, 0, 2], [[0, 1], [2, 3], [4, 5]], 6, 9, keep_all)
    check([0], [1], [[0, 1]], 6, 0, keep_all)
    check([], [], np.zeros((0, 2), np.int64), 6, 5, keep_all)


def test_requests_that_cannot_run(cuda_device):
    """Each kind alone: skipped, recorded, the others untouched."""
    base = dict(lens=[2, 1, 2], kept=[1, 2, 0], table=[[0, 1], [2, 3], [4, 5]])
    for keep_all in (True, False):
        for change in (dict(kept=[1, 3, 0]), dict(kept=[1, -1, 0]), dict(lens=[2, -4, 2]),
                       dict(table=[[0, 1], [6, 6], [4, 5]]), dict(table=[[0, 1], [-1, -1], [4, 5]]),
                       dict(table=[[0, 1], [2, 2**31 - 1], [4, 5]])):
            d = dict(base, **change)
            check(d["lens"], d["kept"], d["table"], 6, 8, keep_all)
    check([2, 3, 2], [1, 1, 0], base["table"], 6, 8, True)   # more states than slots
    check([2, 1, 2], [1, 1, 0], base["table"], 6, 4, True)   # the last one does not fit
    check([2, 1, 2], [1, 1, 0], base["table"], 6, 1, False)  # only a part of the first fits
    check([2, 1, 2], [1, 1, 0], base["table"], 0, 8, True)   # no pool at all


def test_lengths_beyond_32_bits_in_sum(cuda_device):
    big = 2**31 - 1
    check([1, big, big, big, 2], [0] * 5, [[i] for i in range(5)], 5, 7, False)


def test_table_rows_apart_and_own_outputs(cuda_device):
    lens, kept, table, slots = batch(300, 3, seed=8)
    wide = torch.full((300, 10), -7, dtype=torch.int32, device="cuda")
    wide[:, 2:5] = torch.tensor(table, dtype=torch.int32, device="cuda")
    n = int(lens.sum()) + 11
    out = {k: torch.full((m,), 99, dtype=torch.int32, device="cuda")
           for k, m in (("cu_seqlens", 301), ("src", 300), ("request", n), ("dst", n))}
    got = check(lens, kept, table, slots, n, True, device_table=wide[:, 2:5], out=out)
    assert got is out


def test_captured_with_lengths_written_on_the_gpu(cuda_device):
    """One capture serves every step: lengths and kept counts change in place."""
    lens, kept, table, slots = batch(20, 4, seed=9)
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    l, k, t = dev(lens), dev(kept), dev(table)
    binding.slot_map(l, k, t, slots, 80)  # (the library looks its status word up outside a capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.slot_map(l, k, t, slots, 80)
    for seed in (10, 11):
        lens, kept, _, _ = batch(20, 4, seed=seed)
        l.copy_(dev(lens))
        k.copy_(dev(kept))
        graph.replay()
        torch.cuda.synchronize()
        want = layer.slot_map(lens, kept, table, slots, 80, True)
        for name, w in zip(("cu_seqlens", "src", "request", "dst"), want):
            np.testing.assert_array_equal(got[name].cpu().numpy(), w, err_msg=name)
    assert binding.device_status() == 0
