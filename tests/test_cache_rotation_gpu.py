"""The rotation of dsa_cache_write behind a rounding to bf16 (the last 64 dims
of MODEL1 and V3.2 records), over many rows: every stored value is that of the
rotation in 64 bits, rounded to fp32 and then to bf16.

Without a norm the kernel's rotation is the 64-bit one but for errors of 2^-47
of the products, 2^-23 of an fp32 step: none of four million values may differ.
With one the row's factor is off by up to 2^-26, which moves a value over a
tie of bf16 (steps of 2^-8 to 2^-7 of the value) for at most one in 2^16.5."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def rotated(x, table, style):
    c, s = table[:, :32], table[:, 32:]
    r = x[:, -64:]
    if style == W.ROPE_NEOX:
        a, b = r[:, :32], r[:, 32:]
        return torch.cat([a * c - b * s, b * c + a * s], 1)
    a, b = r[:, 0::2], r[:, 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(1)


@pytest.mark.parametrize("fmt", [W.FMT_MODEL1_584, W.FMT_V32_656])
@pytest.mark.parametrize("style", [W.ROPE_NEOX, W.ROPE_GPTJ])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bf16_dims(fmt, style, norm, dtype):
    n, rb = 65536, W.RECORD_BYTES[fmt]
    d = 576 if fmt == W.FMT_V32_656 else 512
    g = torch.Generator(device="cuda").manual_seed(10 * fmt + style)
    x = torch.randn((n, d), generator=g, device="cuda").to(dtype)
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda") if norm else None
    cs = W.rope_table(W.ROPE_TABLE_ROWS, "cuda")
    pos = torch.randint(0, W.ROPE_TABLE_ROWS, (n,), generator=g, device="cuda")
    cache = W.PagedCache(torch.zeros((n // 64, 64 * rb), dtype=torch.uint8, device="cuda"), 64, fmt)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots, x, norm_weight=w, norm_eps=1e-6, positions=pos, cos_sin=cs, rope_style=style)
    at = 448 if fmt == W.FMT_MODEL1_584 else 528
    got = cache.data.view(n, rb)[:, at:at + 128].contiguous().view(torch.bfloat16)
    v = x.double()
    if norm and fmt == W.FMT_MODEL1_584:     # (a V3.2 row's last 64 dims are not normed)
        v = v * w.double() / (v.square().mean(1, keepdim=True) + float(torch.tensor(1e-6, dtype=torch.float32))).sqrt()
    want = rotated(v, cs[pos].double(), style)
    wrong = int((got != want.float().to(torch.bfloat16)).sum())
    assert wrong <= (n * 64 * 2.0 ** -16.5 if norm and fmt == W.FMT_MODEL1_584 else 0), wrong


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
@pytest.mark.parametrize("style", [W.ROPE_NEOX, W.ROPE_GPTJ])
def test_infinities_and_zeros_in_the_rotated_dims(fmt, style):
    d = 576 if fmt == W.FMT_V32_656 else 512
    x = torch.zeros((3, d), device="cuda")
    x[1] = torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x[2, d - 64] = float("inf")
    cs = W.rope_table(16, "cuda")
    cache = W.PagedCache(torch.zeros((1, 64 * W.RECORD_BYTES[fmt]), dtype=torch.uint8, device="cuda"), 64, fmt)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots, x, positions=torch.tensor([3, 5, 1], device="cuda"), cos_sin=cs, rope_style=style)
    out = torch.empty((3, d), device="cuda")
    B.dsa_cache_read(cache, slots, out)
    assert bool((out[0] == 0).all()) and bool(torch.isfinite(out[1]).all())
    pair = [d - 64, d - 32 if style == W.ROPE_NEOX else d - 63]      # (inf c, inf s), c and s > 0 at position 1
    if fmt in (W.FMT_MODEL1_584, W.FMT_V32_656):                     # bf16
        assert bool((out[2, pair] == float("inf")).all()) and bool((out[2, :d - 64] == 0).all())
    elif fmt == W.FMT_FP8_528:                                       # its block reads back as NaN
        assert bool(torch.isnan(out[2, 384:]).all()) and bool((out[2, :384] == 0).all())
    else:                                                            # the scale saturates
        assert bool((out[2, pair] > 1e3).all())
