"""The RMS norm of dsa_cache_write at the ends of its range: rows from the
smallest to the largest finite values, whose squares no 32-bit number holds,
and rows of zeros. Values read back against the 64-bit formula, within the
format's rounding (tests/_cache_ref.py) and the fp32 transform's 2^-20."""
import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import _cache_ref as R
from tests.test_cache_gpu import FORMATS, dims, empty_cache, records

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1e30])
def test_rows_of_any_magnitude(fmt, dtype, eps):
    exps = [-125, -120, -100, -80, -70, -64, -63, -62, -50, -31, -30, -29, -10, 0, 30, 49, 50, 51, 60, 63, 64, 65, 100, 126]
    n = len(exps)
    g = torch.Generator().manual_seed(5)
    x = torch.randn((n, dims(fmt)), generator=g, dtype=torch.float64).clamp(-1.9, 1.9)
    x[:, :512] *= torch.exp2(torch.tensor(exps, dtype=torch.float64))[:, None]
    x[:, ::7] *= 2.0 ** -6
    x = x.to(dtype)
    w = 1 + 0.2 * torch.randn(512, generator=g)
    src = R.transform(x.double().numpy(), w.numpy(), float(np.float32(eps)))
    cache = empty_cache(fmt, 64, 64)
    B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), x.cuda(), norm_weight=w.cuda(), norm_eps=eps)
    got = R.record_values(fmt, records(cache)[:n])
    # (values below 2^-110 lie among the products' subnormals)
    tol = R.quant_bound(fmt, src) * (1 + 2.0 ** -10) + np.abs(src) * 2.0 ** -20 + 2.0 ** -133
    tol = np.where(np.abs(src) < 2.0 ** -110, np.abs(src) + 2.0 ** -110, tol)
    err = np.abs(got - src)
    bad = np.argwhere(~(err <= tol))
    assert bad.size == 0, [(exps[i], int(j), float(got[i, j]), float(src[i, j])) for i, j in bad[:5]]


@pytest.mark.parametrize("fmt", FORMATS)
def test_zero_rows(fmt):
    """x / sqrt(0 + eps): zeros, and 0 / 0 with eps = 0."""
    x = torch.zeros((3, dims(fmt)))
    x[1] = torch.randn(dims(fmt), generator=torch.Generator().manual_seed(1))
    w = torch.ones(512, device="cuda")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, dims(fmt)), device="cuda")
    cache = empty_cache(fmt, 64, 64)
    B.dsa_cache_write(cache, slots, x.cuda(), norm_weight=w, norm_eps=1e-6)
    B.dsa_cache_read(cache, slots, out)
    assert bool((out[[0, 2]] == 0).all()) and bool(torch.isfinite(out).all())
    B.dsa_cache_write(cache, slots, x.cuda(), norm_weight=w, norm_eps=0.0)
    again = torch.empty_like(out)
    B.dsa_cache_read(cache, slots, again)
    assert bool(torch.isnan(again[[0, 2], :512]).all()) and bool(torch.isfinite(again[1]).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nonfinite_rows_with_the_norm(fmt):
    """A NaN makes the whole row NaN; with an infinity the mean is infinite,
    its own value inf / inf and every other one zero."""
    x = torch.randn((3, dims(fmt)), generator=torch.Generator().manual_seed(2))
    x[0, 9] = float("nan")
    x[1, 9] = float("inf")
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, dims(fmt)), device="cuda")
    cache = empty_cache(fmt, 64, 64)
    B.dsa_cache_write(cache, slots, x.cuda(), norm_weight=torch.ones(512, device="cuda"), norm_eps=1e-6)
    B.dsa_cache_read(cache, slots, out)
    assert bool(torch.isnan(out[0, :512]).all()) and bool(torch.isfinite(out[2]).all())
    size = R.block_dims(fmt)
    assert bool(torch.isnan(out[1, :size]).all()) and bool((out[1, size:512] == 0).all())
