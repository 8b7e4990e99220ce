"""dsa_weights_run of a step without tokens: the lists' scores arrive in scores_out
all the same, and what lies behind the lists' ends is left as it was."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests._serve_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def empty(fmt, lengths, width):
    return Batch([(0, n) for n in lengths], 16, fmt, width=width, seed=3)


def run(c, before, out, attn=None, **kw):
    attn = attn or B.AttentionWeights(0, c.B, c.H, c.width, "cuda", c.d)
    lse = torch.empty((0, c.H), device="cuda")
    assert c.q.shape[0] == 0
    attn(c.q, c.cache, c.slots, c.lengths, c.starts, lse, before, out, c.scale, c.window, c.sink, **kw)
    return attn


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_V32_656])
@pytest.mark.parametrize("base", [False, True])
@pytest.mark.parametrize("lengths,width", [([30, 0, 200], 200), ([-4, 1 << 20, 7], 128), ([5000, 4096, 4097, 1], 5001), ([1], 1)])
def test_scores_arrive(fmt, base, lengths, width):
    c = empty(fmt, lengths, width)
    before = torch.rand((c.B, width), device="cuda") if base else None
    out = torch.full((c.B, width), 7.0, device="cuda")
    attn = run(c, before, out)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == 0
    for b, n in enumerate(lengths):
        n = min(max(n, 0), width)
        assert torch.equal(out[b, :n], torch.zeros(n, device="cuda") if before is None else before[b, :n])
        assert bool((out[b, n:] == 7).all())


def test_in_place_keeps_the_scores():
    c = empty(W.FMT_FP8_528, [30, 200], 200)
    scores = torch.rand((2, 200), device="cuda")
    want = scores.clone()
    run(c, scores, scores)
    torch.cuda.synchronize()
    assert torch.equal(scores, want)


def test_starts_that_do_not_ascend_write_nothing():
    c = empty(W.FMT_FP8_528, [30, 200], 200)
    c.starts[1] = 1
    out = torch.full((2, 200), 7.0, device="cuda")
    attn = run(c, None, out)
    assert B.dsa_decode_read_status(attn.workspace) == -1
    assert bool((out == 7).all())
    c.starts[1] = 0
    run(c, None, out, attn)
    assert B.dsa_decode_read_status(attn.workspace) == 0
    assert bool((out[0, :30] == 0).all()) and bool((out[1] == 0).all())


def test_captured_and_on_another_stream():
    c = empty(W.FMT_FP8_528, [30, 0, 200], 200)
    before, out = torch.rand((3, 200), device="cuda"), torch.full((3, 200), 7.0, device="cuda")
    attn = run(c, before, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(c, before, out, attn)
    c.lengths.copy_(torch.tensor([150, 3, 0]))
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    for b, n in enumerate([150, 3, 0]):
        assert torch.equal(out[b, :n], before[b, :n]) and bool((out[b, n:] == 7).all())
    st = torch.cuda.Stream()
    out.fill_(7.0)
    torch.cuda.synchronize()
    run(c, before, out, attn, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out[0, :150], before[0, :150])
