"""dsa_weights_run: the scores of entries that no token sees, on their way from one
array to another in pieces of a list."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import test_weights_gpu as WT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("sms", [2, 0])
@pytest.mark.parametrize("window", [1, 128])
def test_long_lists_that_a_window_leaves(window, sms):
    c = WT.Case([(1, 40000), (2, 4096), (0, 9000), (3, 4097), (1, 12289)], 16, W.FMT_FP8_528, seed=7, width=40001, window=window,
                num_slots=8192)
    c.check(c.run(sms)[0])
