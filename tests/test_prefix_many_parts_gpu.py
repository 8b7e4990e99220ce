"""The shared-prefix merge over more parts than it holds weights for at a time:
one row tile cut over hundreds of CTA pairs (num_sms past the device's)."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests.test_prefix_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("sms,pairs", [(512, 256), (516, 258), (1400, 274)])
@pytest.mark.parametrize("tail", [False, True])
def test_parts_past_one_round(sms, pairs, tail):
    c = Case(3, 8, 70000, W.FMT_NVFP4_288, seed=51, num_slots=4096, sink=True, tail=tail, invalid=0.02)
    out, lse, attn = c.run(num_sms=sms)
    assert attn.plan.pairs == pairs and attn.plan.row_tiles == 1
    c.check(out, lse)


def test_nan_and_empty_parts_past_one_round():
    c = Case(2, 8, 150000, W.FMT_NVFP4_288, seed=52, num_slots=4096)
    c.slots[:140000] = -1                    # the kept keys in the last of three rounds
    out, lse, attn = c.run(num_sms=1200)
    assert attn.plan.pairs == 586
    c.check(out, lse)
    c.cache.data[:, :64 * 288].view(-1, 64, 288)[0, 5, 256:288] = 0x7F     # slot 5: NaN scales
    c.slots[:] = -1
    c.slots[-1] = 5
    c.slots[:100] = 9
    out, lse, _ = c.run(num_sms=1200)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
