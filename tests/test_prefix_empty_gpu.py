"""dsa_prefix_run where the prefix keeps nothing: lists of every length up to
one key tile, both key sizes, with and without a tail, in a workspace cut from
the middle of a larger buffer whose rest stays as it was."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests.test_prefix_gpu import Case

pytestmark = pytest.mark.gpu
MARGIN = 1 << 20


@pytest.fixture(scope="module", autouse=True, params=[False, True], ids=["release", "checking"])
def lib(request):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    BLD.build(debug=True)
    B.load()
    B.use_checking_build(request.param)
    yield
    B.use_checking_build(False)


def in_the_middle(T, H, width, d, num_sms=0):
    attn = B.PrefixAttention(T, H, width, "cuda", d, num_sms)
    n = attn.workspace.numel()
    whole = torch.full((n + 2 * MARGIN,), 0xA5, dtype=torch.uint8, device="cuda")
    attn.workspace = whole[MARGIN:MARGIN + n]
    assert attn.workspace.data_ptr() % 256 == 0
    return attn, whole


def margins_untouched(whole):
    return bool((whole[:MARGIN] == 0xA5).all()) and bool((whole[-MARGIN:] == 0xA5).all())


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_V32_656])
@pytest.mark.parametrize("width", [1, 200, 256])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("what", [0, -3, "no slot kept"])
@pytest.mark.parametrize("T,H", [(1, 8), (33, 64)])
def test_nothing_kept(fmt, width, tail, what, T, H):
    length = width if isinstance(what, str) else what
    c = Case(T, H, width, fmt, seed=width, length=length, sink=True, tail=tail)
    if isinstance(what, str):
        c.slots.fill_(-1)
    attn, whole = in_the_middle(T, H, width, c.d)
    out, lse, _ = c.run(attn=attn)           # (status 0: no check fires)
    c.check(out, lse)
    assert margins_untouched(whole)
    c.length.fill_(1)                        # the same plan with a key again
    c.slots.fill_(3)
    out, lse, _ = c.run(attn=attn)
    c.check(out, lse)
    assert margins_untouched(whole)


def test_captured_call_whose_length_becomes_zero():
    c = Case(4, 16, 256, W.FMT_FP8_528, seed=3, sink=True, tail=True)
    attn, whole = in_the_middle(4, 16, 256, c.d)
    call = lambda: attn(c.q, c.cache, c.slots, c.length, c.scale, c.sink, None, None, 0, c.tail_out, c.tail_lse)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for length in (256, 0, 100, -1):
        c.length.fill_(length)
        attn.out.fill_(float("nan"))
        attn.lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert B.dsa_decode_read_status(attn.workspace) == 0
        c.check(attn.out, attn.lse)
    assert margins_untouched(whole)
