"""dsa_chunk_run with row tiles that have no keys (a list of length 0, or one
shorter than its chunk by 128 rows and more) between others of the same CTA pair,
against the formulas in 64 bits and the tolerances of test_chunk_gpu."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import test_chunk_gpu as CH
from tests._serve_ref import Batch

pytestmark = pytest.mark.gpu
FORMATS = list(W.RECORD_BYTES)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def table(fmt, rope):
    return None if fmt == W.FMT_V32_656 else rope


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("rope", [None, W.ROPE_NEOX])
@pytest.mark.parametrize("sizes,H", [([(1, 200), (1, 0), (1, 200)], 64), ([(4, 300), (4, 0), (4, 300)], 32),
                                     ([(4, 300), (12, 4), (2, 300)], 32), ([(5, 300), (9, 0), (3, 2), (0, 7), (7, 290)], 20)])
def test_one_pair(fmt, tail, rope, sizes, H):
    c = Batch(sizes, H, fmt, seed=fmt, width=320, sink=True, tail=tail, rope=table(fmt, rope))
    CH.check(c, *CH.run(c, 2)[:2])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("idle", [(80,), (0, 1, 2, 77, 78, 159), tuple(range(1, 160, 3))])
def test_idle_requests_among_single_tokens(fmt, tail, idle):
    sizes = [(1, 0 if b in idle else 40 + b % 89) for b in range(160)]
    c = Batch(sizes, 64, fmt, seed=9, width=128, sink=True, tail=tail, rope=table(fmt, W.ROPE_GPTJ))
    CH.check(c, *CH.run(c)[:2])


@pytest.mark.parametrize("window", [0, 128])
@pytest.mark.parametrize("sms", [2, 6, 0])
def test_chunks_past_the_start_of_their_lists(window, sms):
    """Tiles whose rows all lie before the list's first entry, or some of them."""
    c = Batch([(30, 500), (40, 11), (1, 128), (70, 33), (20, 20), (33, 400)], 64, W.FMT_FP8_528_UE8M0, seed=10, width=512,
              sink=True, rope=W.ROPE_NEOX, window=window)
    CH.check(c, *CH.run(c, sms)[:2])
