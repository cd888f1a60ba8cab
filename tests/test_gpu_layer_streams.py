"""Memory of the calls that run on another stream than the current one (stream=)."""
import pytest
import torch

from gated_delta_rule_93_b200 import binding

pytestmark = pytest.mark.gpu

ROWS, G, D = 8192, 16, 128  # a 64 MB dx: blocks of this size are the allocator's own
PASSES = 400                # over 64 MB, in order: several milliseconds


def span(t):
    return t.data_ptr(), t.data_ptr() + t.nbytes


def apart(a, b):
    """Whether two spans share no byte."""
    return a[1] <= b[0] or b[1] <= a[0]


def long_chain(t):
    """t + PASSES in place, one ordinary kernel after the other on the current stream."""
    for _ in range(PASSES):
        t.add_(1.0)


@pytest.fixture
def batch(cuda_device):
    gen = torch.Generator().manual_seed(31)
    x = torch.randn(ROWS, G, D, generator=gen).cuda()
    w = torch.randn(D, generator=gen).cuda()
    want = binding.group_norm_bwd(x, x, x, w)
    torch.cuda.synchronize()
    return x, w, want


def test_outputs_are_not_memory_that_the_current_stream_still_uses(batch):
    """Blocks freed on the current stream while a long chain of kernels queued there
    still works on them: a call on another stream must not be given them."""
    x, w, want = batch
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        blocks = [torch.zeros(ROWS, G, D, device="cuda") for _ in range(3)]
        spans = [span(t) for t in blocks]
        for t in blocks:
            long_chain(t)
        keep = [t.clone() for t in blocks]
        del blocks, t  # free for this stream, whose kernels have not run yet
        got = binding.group_norm_bwd(x, x, x, w, stream=side)
        for name in ("dx", "dz", "dweight"):
            assert all(apart(span(got[name]), s) for s in spans), name
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(got[n], want[n]) for n in ("dx", "dz", "dweight"))
        assert all(bool((t == PASSES).all()) for t in keep)
        del got, keep


def test_outputs_stay_while_the_current_stream_reads_them(batch):
    """An output freed while the current stream still works on it is not handed to the
    next call on the call's own stream."""
    x, w, want = batch
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = binding.group_norm_bwd(x, x, x, w, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        dx = got["dx"]
        long_chain(dx)
        keep = dx.clone()
        freed = span(dx)
        del got, dx
        again = binding.group_norm_bwd(x, x, x, w, stream=side)
        assert all(apart(span(again[n]), freed) for n in ("dx", "dz"))
        torch.cuda.current_stream().wait_stream(side)
        expect = want["dx"].clone()
        long_chain(expect)
        assert torch.equal(keep, expect) and torch.equal(again["dx"], want["dx"])
        del again, keep, expect


@pytest.mark.parametrize("op", ["step", "map", "norm", "prologue", "prologue gradient"])
def test_every_entry_point_allocates_for_its_stream(cuda_device, op):
    """What a call on another stream returns lies in no block that was freed on the current
    stream just before, whatever its size."""
    n = lambda *s: torch.randn(*s, device="cuda")
    q, v, a, s = n(512, 2, 64), n(512, 4, 64), n(512, 4), n(4).abs()
    i = torch.arange(512, dtype=torch.int32, device="cuda")
    pool, up = n(512, 4, 64, 64), n(512, 4, 64)
    one = torch.ones_like(i)
    run = {
        "step": lambda **k: [binding.step_slots(q, q, v, a, a, pool, i, gate_scale=s, norm_q=True,
                                                norm_k=True, **k)],
        "map": lambda **k: binding.slot_map(one, one, i[:, None], 512, 700, **k).values(),
        "norm": lambda **k: [binding.group_norm_fwd(v, **k)],
        "prologue": lambda **k: binding.prologue_fwd(q, q, a, a, s, **k),
        "prologue gradient": lambda **k: binding.prologue_bwd(q, q, a, a, s, up, up, a, a,
                                                              **k).values()}[op]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    first = list(run())
    torch.cuda.synchronize()
    spans = [span(t) for t in first]
    del first  # blocks of just these sizes are free on the current stream
    got = list(run(stream=side))
    for t in got:
        assert all(apart(span(t), s) for s in spans)
    side.synchronize()


def test_captured_on_a_stream_of_its_own(batch):
    """A call on a stream that joins a capture: its memory is the graph's."""
    x, w, want = batch
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        got = binding.group_norm_bwd(x, x, x, w, stream=side)
        now.wait_stream(side)
        double = got["dx"] * 2
    for _ in range(2):
        junk = torch.full((ROWS, G, D), float("nan"), device="cuda")
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in ("dx", "dz", "dweight"))
        assert torch.equal(double, want["dx"] * 2) and torch.isnan(junk).all()


@pytest.mark.parametrize("captured", [False, True])
def test_events_of_other_streams_are_waited_for(batch, captured):
    """Kernels that are set up while the one before them on their stream ends wait all the
    same for an event of another stream that lies between the two."""
    x, w, _ = batch
    start = x.clone()
    for _ in range(PASSES):
        start.add_(1.0)
    first, want = binding.group_norm_fwd(x, None, w), binding.group_norm_fwd(start, None, w)
    q, a, s = x.view(-1, 16, 128)[:, :2], torch.zeros(ROWS, 16, device="cuda"), torch.ones(16, device="cuda")
    want_q = binding.prologue_fwd(start[:, :2], start[:, :2], a, a, s)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = x.clone()

    def work():
        now = torch.cuda.current_stream()
        side.wait_stream(now)
        y0 = binding.group_norm_fwd(x, None, w, stream=side)  # (of x as it was)
        now.wait_stream(side)
        long_chain(x)
        y1 = binding.group_norm_fwd(start, None, w, stream=side)  # a kernel right before
        side.wait_stream(now)
        y2 = binding.group_norm_fwd(x, None, w, stream=side)
        side.wait_stream(now)
        y3 = binding.prologue_fwd(q, q, a, a, s, stream=side)[0]
        now.wait_stream(side)
        return y0, y1, y2, y3

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = work()
        for _ in range(2):
            x.copy_(keep)
            graph.replay()
    else:
        got = work()
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(got, (first, want, want, want_q)))
