"""Finite keys of any scale: records whose scales are large and whose codes are
small stay within the range that the calls state (largest magnitude up to 2^48),
against the formulas in 64 bits and the tolerances of test_chunk_gpu and
test_weights_gpu."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import test_chunk_gpu as CH
from tests import test_weights_gpu as WT
from tests._serve_ref import Batch

pytestmark = pytest.mark.gpu
SCALED = [W.FMT_FP8_528, W.FMT_FP8_528_UE8M0, W.FMT_MODEL1_584, W.FMT_V32_656]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def rewrite(c, k, every=1):
    """Every `every`th record: codes of 1 to 7 times 2^-9, scales 2^k, bf16 parts
    of the same magnitude."""
    g = torch.Generator(device="cuda").manual_seed(k)
    rec = c.cache.data[:, :c.cache.page_size * c.cache.record_bytes].view(-1, c.cache.page_size, c.cache.record_bytes)
    rec = rec.reshape(-1, c.cache.record_bytes)[::every]   # (a copy: put back below)
    n, codes = len(rec), 448 if c.fmt == W.FMT_MODEL1_584 else 512
    rec[:, :codes] = (torch.randint(1, 8, (n, codes), generator=g, device="cuda") |
                      (torch.randint(0, 2, (n, codes), generator=g, device="cuda") << 7)).to(torch.uint8)
    if c.fmt in (W.FMT_FP8_528, W.FMT_V32_656):
        rec[:, 512:528] = torch.full((n, 4), 2.0 ** k, device="cuda").view(torch.uint8)
    elif c.fmt == W.FMT_FP8_528_UE8M0:
        rec[:, 512:528] = 127 + k
    else:
        rec[:, 576:583] = 127 + k
    at = {W.FMT_MODEL1_584: 448, W.FMT_V32_656: 528}.get(c.fmt)
    if at:
        part = (torch.rand((n, 64), generator=g, device="cuda") - 0.5) * 2.0 ** (k - 7)
        rec[:, at:at + 128] = part.to(torch.bfloat16).view(torch.uint8)
    whole = c.cache.data[:, :c.cache.page_size * c.cache.record_bytes].reshape(-1, c.cache.record_bytes)
    whole[::every] = rec
    c.cache.data[:, :c.cache.page_size * c.cache.record_bytes] = whole.view(c.cache.data.shape[0], -1)


def batch(fmt, k, every=1):
    c = Batch([(20, 300), (1, 257), (3, 70)], 32, fmt, seed=fmt + k, sink=True, q_log2=7 - k, window=200)
    rewrite(c, k, every)
    return c


@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("k", [30, 41, 54])
def test_chunk(fmt, k):
    c = batch(fmt, k)
    CH.check(c, *CH.run(c)[:2])


@pytest.mark.parametrize("fmt", SCALED)
@pytest.mark.parametrize("k", [30, 41, 54])
def test_weights(fmt, k):
    case = WT.Case.__new__(WT.Case)
    case.c = c = batch(fmt, k)
    case.lse = torch.full((c.T, c.H), -float("inf"), dtype=torch.float64, device="cuda")
    for b, t, at, key, x, mass in c.scores():
        case.lse[t:t + x.shape[0]] = torch.logsumexp(x, 2)
    case.lse, case.before = case.lse.float(), None
    case.check(case.run()[0])


@pytest.mark.parametrize("fmt", SCALED)
def test_chunk_among_ordinary_keys(fmt):
    """One exponent per key where a group's magnitudes differ."""
    c = Batch([(20, 300), (1, 257)], 32, fmt, seed=fmt, q_log2=-34)
    rewrite(c, 41, every=7)
    CH.check(c, *CH.run(c)[:2])


@pytest.mark.parametrize("fmt", SCALED)
def test_key_past_the_range_stays_where_it_is_seen(fmt):
    """An element of 2^49 or more makes the scores of its key NaN."""
    c = Batch([(40, 300)], 16, fmt, seed=17, window=20)
    c.slots[c.slots == 0] = -1
    c.slots[0, 270] = 0                      # the position of token 10
    rec = c.cache.data[0, :c.cache.record_bytes]
    rec[3] = 0x08                            # 2^-6
    if fmt in (W.FMT_FP8_528, W.FMT_V32_656):
        rec[512:516].view(torch.float32).fill_(2.0 ** 60)
    else:
        rec[512 if fmt == W.FMT_FP8_528_UE8M0 else 576] = 127 + 60
    out, lse, _ = CH.run(c)
    sees = torch.zeros(40, dtype=torch.bool, device="cuda")
    sees[10:30] = True
    assert bool(torch.isnan(lse[sees]).all()) and bool(torch.isnan(out[sees]).all())
    assert bool(torch.isfinite(lse[~sees]).all()) and bool(torch.isfinite(out[~sees]).all())
