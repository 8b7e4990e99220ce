"""The prompt calls in the checking build: no check fires on real extents and
the results are those of the release build's tests; with the extent narrowed (a
knob of the checking build) the records past it are reported and skipped."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import test_chunk_gpu as CH
from tests import test_weights_gpu as WT
from tests._serve_ref import Batch
from tests.test_evict_gpu import Lists
from tests.test_qk_gpu import check, empty, make, reference

pytestmark = pytest.mark.gpu
DSA_ERR_BOUNDS = -8


@pytest.fixture(scope="module", autouse=True)
def checking_build():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    BLD.build(debug=True)
    B.load()
    B.use_checking_build(True)
    yield
    B.use_checking_build(False)


SIZES = ([(1, 1)], [(33, 700), (1, 513), (0, 90), (90, 612)], [(150, 400)])


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
@pytest.mark.parametrize("window", [0, 70])
def test_no_check_fires(fmt, window):
    for sizes in SIZES:
        c = Batch(sizes, 20, fmt, seed=fmt, sink=True, tail=True, invalid=0.05, window=window)
        CH.check(c, *CH.run(c)[:2])
        w = WT.Case(sizes, 64, fmt, seed=fmt, sink=True, window=window)
        w.check(w.run()[0])


def test_narrowed_extent(monkeypatch):
    c = Batch([(20, 300), (3, 200)], 16, W.FMT_FP8_528, seed=3)
    w = WT.Case([(20, 300), (3, 200)], 16, W.FMT_FP8_528, seed=3)
    monkeypatch.setenv("DSA_DEBUG_CHECK_EXTENT", str(c.cache.data.numel() // 2))
    attn = CH.attention(c)
    attn.out.fill_(7.0)
    CH.call(c, attn)
    assert B.dsa_decode_read_status(attn.workspace) == DSA_ERR_BOUNDS
    weights = B.AttentionWeights(w.c.T, w.c.B, 16, w.c.width, "cuda")
    sums = torch.full((2, 300), 7.0, device="cuda")
    w.call(weights, sums)
    assert B.dsa_decode_read_status(weights.workspace) == DSA_ERR_BOUNDS
    for b in (c, w.c):                       # those records were not kept
        b.slots[b.slots >= b.cache.num_slots // 2] = -1
    CH.check(c, attn.out, attn.lse)
    w.check(sums)


def test_norm_and_eviction():
    for fmt in W.RECORD_BYTES:
        q, k, qw, kw, slots, args = make(9, 20, fmt, torch.bfloat16, fmt)
        out, cache, same = torch.empty_like(q), empty(fmt, 14), empty(fmt, 14)
        B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, **args)
        B.dsa_cache_write(same, slots, k, kw, 1e-6, args["positions"], args["cos_sin"])
        torch.cuda.synchronize()
        check(out, *reference(q, qw, 1e-6, args["positions"], args["cos_sin"], 0))
        assert torch.equal(cache.data, same.data)
    c = Lists([2000, 301, 300, 2047], 2047, 300, 4, 32)
    c.call()
    c.check()
