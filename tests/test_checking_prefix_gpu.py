"""The cache calls and the shared-prefix attention in the checking build: no
record check fires on real extents and the results are those of the release
build's tests; with the extent narrowed (the knob of the checking build) the
records past it are reported and skipped, never touched."""
import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests.test_cache_gpu import ENC, draw_rows, empty_cache, records
from tests.test_prefix_gpu import Case

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


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
def test_prefix_no_check_fires(fmt):
    for T, H, width in ((1, 1, 1), (3, 20, 300), (20, 32, 700)):
        c = Case(T, H, width, fmt, seed=fmt + T, sink=True, tail=True, invalid=0.05)
        out, lse, _ = c.run()
        c.check(out, lse)


def test_prefix_record_check_fires_and_skips(monkeypatch):
    c = Case(2, 16, 300, W.FMT_FP8_528, seed=3)
    monkeypatch.setenv("DSA_DEBUG_CHECK_EXTENT", str(c.cache.data.numel() // 2))
    attn = B.PrefixAttention(2, 16, 300, "cuda")
    attn(c.q, c.cache, c.slots, c.length, c.scale)
    assert B.dsa_decode_read_status(attn.workspace) == DSA_ERR_BOUNDS
    assert int(attn.workspace[4:8].view(torch.int32).item()) == 1      # kind: a record read
    half = c.slots.clone()
    half[half >= c.cache.num_slots // 2] = -1
    c.slots = half                                                     # those rows were not kept
    c.check(attn.out, attn.lse)
    monkeypatch.delenv("DSA_DEBUG_CHECK_EXTENT")
    out, lse, _ = c.run(attn=attn)
    c.check(out, lse)


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
def test_cache_calls(fmt, monkeypatch):
    n, num = 70, 128
    x = draw_rows(n, fmt, torch.bfloat16, fmt)
    slots = torch.randperm(num, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32)
    want = ENC[fmt](x.float()).numpy()
    cache = empty_cache(fmt, num, 64)
    B.dsa_cache_write(cache, slots.cuda(), x.cuda())
    assert np.array_equal(records(cache)[slots.numpy()], want)
    monkeypatch.setenv("DSA_DEBUG_CHECK_EXTENT", str(cache.data.numel() // 2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = empty_cache(fmt, num, 64)
    B.dsa_cache_write(cache, slots.cuda(), x.cuda(), device_status=status)
    assert int(status) == DSA_ERR_BOUNDS
    got, low = records(cache), slots.numpy() < num // 2
    assert np.array_equal(got[slots.numpy()[low]], want[low]) and np.all(got[num // 2:] == 0xA5)
    out = torch.empty((n, x.shape[1]), device="cuda")
    B.dsa_cache_read(cache, slots.cuda(), out)
    assert bool((out[torch.from_numpy(~low).cuda()] == 0).all())
