"""Shared-prefix attention over records that hold blocks of zeros: a block's
scale byte (2^0 for zeros) says nothing about a key whose codes are all zero,
so small keys keep their precision and zero keys do not send their group of 32
to the path with one exponent per key. Against the formulas in 64 bits, with
the tolerances of test_prefix_gpu."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests.test_prefix_gpu import Case

pytestmark = pytest.mark.gpu
FORMATS = list(W.RECORD_BYTES)
MIXED = -2 ** 31


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def case_of(fmt, rows, q_log2=0):
    """A case whose list names the given rows, in their order."""
    n = rows.shape[0]
    c = Case(3, 32, n, fmt, seed=70 + fmt, q_log2=q_log2)
    c.slots = torch.arange(n, dtype=torch.int32, device="cuda")
    c.cache.data.zero_()
    B.dsa_cache_write(c.cache, c.slots, rows.cuda())
    return c


def group_exponents(c, attn):
    at = attn.plan.ws_info_offset
    n = -(-c.width // 32)
    return attn.workspace[at:at + 8 * n].view(torch.int32).view(n, 2)[:, 0]


def draw(fmt, n, log2=0):
    d = 576 if fmt == W.FMT_V32_656 else 512
    return torch.randn((n, d), generator=torch.Generator().manual_seed(fmt)) * 2.0 ** log2


@pytest.mark.parametrize("fmt", [f for f in FORMATS if f != W.FMT_NVFP4_288])   # (its scales end at 2^-9)
@pytest.mark.parametrize("log2", [-26, -30, -34, -45])
def test_small_keys_with_zero_blocks(fmt, log2):
    x = draw(fmt, 300, log2)
    x[:, 64:192] = 0
    x[7, :448] = 0
    x[8, :] = 0
    c = case_of(fmt, x, q_log2=-log2)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_small_nonzero_block_among_zeros(fmt):
    """One block of a key holds all of it, at every place."""
    x = torch.zeros((160, 576 if fmt == W.FMT_V32_656 else 512))
    full = draw(fmt, 160, -3 if fmt == W.FMT_NVFP4_288 else -40)
    for i in range(160):
        a = 16 * (i % (x.shape[1] // 16))
        x[i, a:a + 16] = full[i, a:a + 16]
    c = case_of(fmt, x, q_log2=0 if fmt == W.FMT_NVFP4_288 else 40)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
def test_zeros_among_ordinary_keys_keep_the_groups_exponent(fmt):
    x = draw(fmt, 256, 3)                    # 2^3: away from the exponent that a block of zeros reads as
    x[::5] = 0
    x[1::5, 128:256] = 0
    c = case_of(fmt, x)
    out, lse, attn = c.run()
    c.check(out, lse)
    assert not bool((group_exponents(c, attn) == MIXED).any())


def test_only_zero_keys():
    for fmt in FORMATS:
        c = case_of(fmt, torch.zeros_like(draw(fmt, 70)))
        out, lse, attn = c.run()
        c.check(out, lse)
        assert not bool((group_exponents(c, attn) == MIXED).any())
