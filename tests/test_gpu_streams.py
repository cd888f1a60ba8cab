"""Memory of the mixer's calls that run on another stream than the current one (stream=)."""
import pytest
import torch

from gated_delta_rule_93_b200 import binding

pytestmark = pytest.mark.gpu


def span(t):
    return t.data_ptr(), t.data_ptr() + t.nbytes


def apart(a, b):
    """Whether two spans share no byte."""
    return a[1] <= b[0] or b[1] <= a[0]


def calls():
    gen = torch.Generator().manual_seed(41)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    unit = lambda *s: torch.nn.functional.normalize(n(*s), dim=-1).bfloat16()
    B, T, H, d = 2, 512, 4, 128
    q, k, v = unit(B, T, H, d), unit(B, T, H, d), n(B, T, H, d).bfloat16()
    a, b = n(B, T, H), n(B, T, H)
    g, beta = -0.1 * torch.nn.functional.softplus(a), torch.sigmoid(b)
    flat = [t.flatten(0, 1) for t in (q, k, v, g, beta)]
    cu = torch.tensor([0, 300, B * T], dtype=torch.int32, device="cuda")
    ws = torch.empty(3 * B * 4 * H * d * d * 4, dtype=torch.uint8, device="cuda")
    S, dout = n(B * T, H, d, d), n(B, T, H, d)
    start = S.clone()

    def step(**kw):
        S.copy_(start)
        torch.cuda.synchronize()
        return binding.step(*flat, S, **kw)

    return {
        "chunk_fwd": lambda **kw: binding.chunk_fwd(q, k, v, g, beta, **kw),
        "segmented": lambda **kw: binding.chunk_fwd_segmented(q, k, v, g, beta, segments=4,
                                                              workspace=ws, **kw),
        "varlen": lambda **kw: binding.chunk_fwd_varlen(*flat, cu, **kw),
        "gla": lambda **kw: binding.chunk_fwd_gla(q, k, v, g, **kw),
        "prologue": lambda **kw: binding.chunk_fwd_prologue(q, k, v, a, b, a[0, 0].abs(), **kw),
        "dplr": lambda **kw: binding.dplr_fwd(q, k, v, q, k, g, **kw),
        "backward": lambda **kw: tuple(binding.chunk_bwd(q, k, v, g, beta, dout, **kw).values()),
        "step": lambda **kw: (step(**kw),),
    }


@pytest.mark.parametrize("op", ["chunk_fwd", "segmented", "varlen", "gla", "prologue", "dplr",
                                "backward", "step"])
def test_outputs_are_of_the_calls_own_stream(cuda_device, op):
    """Blocks of just the outputs' sizes are free on the current stream, whose kernels
    still work on them; the call must not be given them, and answers as ever."""
    run = calls()[op]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = run()
    torch.cuda.synchronize()
    want = [t.cpu() for t in want]
    blocks = list(run())
    torch.cuda.synchronize()
    for t in blocks:
        for _ in range(200):
            t.zero_()
    spans = [span(t) for t in blocks]
    del blocks, t
    got = run(stream=side)
    assert all(apart(span(x), s) for x in got for s in spans)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x.cpu(), w) for x, w in zip(got, want))
    assert binding.device_status() == 0


def test_a_long_sequence_keeps_its_workspace(cuda_device):
    """The workspace of a call on another stream is not handed out again before that
    stream is done with it."""
    gen = torch.Generator().manual_seed(42)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()
    T, H, d = 16384, 4, 128
    q, k = (torch.nn.functional.normalize(n(1, T, H, d), dim=-1).bfloat16() for _ in range(2))
    v, g, beta = n(1, T, H, d).bfloat16(), -0.1 * n(1, T, H).abs(), torch.sigmoid(n(1, T, H))
    need = binding.chunk_fwd_workspace_bytes(1, T, H, d, d)
    assert need > 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, S = (t.clone() for t in binding.chunk_fwd(q, k, v, g, beta))
    torch.cuda.synchronize()
    for _ in range(5):
        o1, S1 = binding.chunk_fwd(q, k, v, g, beta, stream=side)
        junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        assert torch.equal(o1, o) and torch.equal(S1, S)
        del junk
