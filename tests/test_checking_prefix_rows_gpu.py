"""The checking build bounds the rows of out, lse and the tail, and the partials
of the shared-prefix attention. Narrowed by the build's knobs
(DSA_DEBUG_CHECK_ROWS, DSA_DEBUG_CHECK_PARTS, read per call) below what is
there, the accesses past them are reported and left out; nothing outside the
real buffers is touched at any time."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests.test_prefix_gpu import Case

pytestmark = pytest.mark.gpu
DSA_ERR_BOUNDS, OUT, PARTIAL = -8, 5, 6


@pytest.fixture(scope="module", autouse=True)
def checking_build():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    BLD.build(debug=True)
    B.load()
    B.use_checking_build(True)
    yield
    B.use_checking_build(False)


def status(attn):
    return B.dsa_decode_read_status(attn.workspace), int(attn.workspace[4:8].view(torch.int32).item())


def call(c, attn):
    attn.out.fill_(7.0)
    attn.lse.fill_(7.0)
    attn(c.q, c.cache, c.slots, c.length, c.scale, c.sink, c.pos, c.cs, c.style, c.tail_out, c.tail_lse)
    torch.cuda.synchronize()


# whole row tiles in a pair; few parts; many parts; no key
SHAPES = [(40, 16, 200, 2, None), (40, 16, 1100, 16, None), (4, 16, 3000, 0, None), (40, 16, 200, 0, 0)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,H,width,sms,length", SHAPES)
def test_output_rows(monkeypatch, T, H, width, sms, length, tail):
    c = Case(T, H, width, W.FMT_FP8_528, seed=90, sink=True, tail=tail, length=length)
    attn = B.PrefixAttention(T, H, width, "cuda", num_sms=sms)
    call(c, attn)
    assert status(attn) == (0, 0)
    c.check(attn.out, attn.lse)
    want, wlse = attn.out.clone().view(-1, 512), attn.lse.clone().view(-1)
    some = T * H // 2 + 3
    monkeypatch.setenv("DSA_DEBUG_CHECK_ROWS", str(some))
    call(c, attn)
    assert status(attn) == (DSA_ERR_BOUNDS, OUT)
    out, lse = attn.out.view(-1, 512), attn.lse.view(-1)
    assert torch.equal(out[:some], want[:some]) and torch.equal(lse[:some], wlse[:some])
    assert bool((out[some:] == 7.0).all()) and bool((lse[some:] == 7.0).all())
    monkeypatch.delenv("DSA_DEBUG_CHECK_ROWS")
    call(c, attn)
    assert status(attn) == (0, 0) and torch.equal(attn.out.view(-1, 512), want)


@pytest.mark.parametrize("T,H,width,sms", [(40, 16, 1100, 16), (4, 16, 3000, 0)])
def test_partial_rows(monkeypatch, T, H, width, sms):
    c = Case(T, H, width, W.FMT_FP8_528, seed=91, sink=True)
    attn = B.PrefixAttention(T, H, width, "cuda", num_sms=sms)
    monkeypatch.setenv("DSA_DEBUG_CHECK_PARTS", "300")
    n = attn.plan.ws_part_o_offset
    attn.workspace[n:] = 0xA5
    call(c, attn)
    assert status(attn) == (DSA_ERR_BOUNDS, PARTIAL)
    parts = attn.workspace[n:].view(-1, 2048)
    assert parts.shape[0] == 256 * attn.plan.pairs and bool((parts[300:] == 0xA5).all())
    assert not bool((parts[:128] == 0xA5).all())
    monkeypatch.delenv("DSA_DEBUG_CHECK_PARTS")
    call(c, attn)
    assert status(attn) == (0, 0)
    c.check(attn.out, attn.lse)


@pytest.mark.parametrize("fmt", [W.FMT_NVFP4_288, W.FMT_V32_656])
def test_no_check_fires(fmt):
    for T, H, width, sms in ((1, 1, 1, 0), (33, 20, 700, 152), (5, 128, 5000, 0), (2, 16, 9000, 1400)):
        c = Case(T, H, width, fmt, seed=92, sink=True, tail=True, invalid=0.05, rope=None if fmt == W.FMT_V32_656 else W.ROPE_GPTJ)
        out, lse, _ = c.run(num_sms=sms)
        c.check(out, lse)
