"""dsa_cache_write / dsa_cache_read on the GPU.

Untransformed rows: the records equal the definition's bit for bit (the
encoders of the workloads module, run on the CPU). Normed and rotated rows:
the values read back lie within the format's own rounding of the 64-bit
transform (tests/_cache_ref.py derives the bound) plus the fp32 transform's
error: 512 squares summed in fp32 pairs, a root, a quotient and two products
stay within 16 half steps of 2^-24 each, taken as 2^-20 of the pair's
magnitudes. Reads: one fp32 product (2^-24) and one rounding to the row type.
"""
import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import _cache_ref as R
from tests._parity import compare, oracle_ref

pytestmark = pytest.mark.gpu
FORMATS = list(W.RECORD_BYTES)
TYPES = [torch.bfloat16, torch.float16, torch.float32]
HALF = {torch.bfloat16: R.EPS_BF16, torch.float16: R.EPS_F16, torch.float32: R.EPS_F32}
ENC = {W.FMT_FP8_528: W.encode_fp8_records, W.FMT_NVFP4_288: W.encode_nvfp4_records,
       W.FMT_FP8_528_UE8M0: W.encode_fp8_ue8m0_records, W.FMT_MODEL1_584: W.encode_model1_records,
       W.FMT_V32_656: W.encode_v32_records}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def dims(fmt):
    return 576 if fmt == W.FMT_V32_656 else 512


def empty_cache(fmt, num_slots, page, pad=0, fill=0xA5):
    data = torch.full((num_slots // page, page * W.RECORD_BYTES[fmt] + pad), fill, dtype=torch.uint8, device="cuda")
    return W.PagedCache(data, page, fmt)


def records(cache):
    rb = cache.record_bytes
    return cache.data[:, :cache.page_size * rb].reshape(-1, rb).cpu().numpy()


def draw_rows(n, fmt, dtype, seed, mag=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, dims(fmt)), generator=g)
    if mag:   # rows and blocks of many magnitudes, a block and a row of zeros
        x = x * torch.exp2(torch.randint(-6, 6, (n, 1), generator=g).float())
        x[:, 64:96] *= 2.0 ** -5
        x[0, 128:256] = 0
        x[n // 2] = 0
    return x.to(dtype)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 5, 257])
def test_write_matches_definition_bit_for_bit(fmt, dtype, n):
    page, num = 16, 512
    x = draw_rows(n, fmt, dtype, 10 * n + fmt)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(num, generator=g)[:n].to(torch.int32)
    if n > 4:
        slots[2], slots[4] = -1, num        # padding, outside
    cache = empty_cache(fmt, num, page, pad=48)
    B.dsa_cache_write(cache, slots.cuda(), x.cuda())
    torch.cuda.synchronize()
    want = np.full((num, cache.record_bytes), 0xA5, np.uint8)
    keep = (slots >= 0) & (slots < num)
    want[slots[keep].long().numpy()] = ENC[fmt](x[keep].float()).numpy()
    got = records(cache)
    bad = np.argwhere(got != want)
    assert bad.size == 0, (bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])
    assert bool((cache.data[:, page * cache.record_bytes:] == 0xA5).all())   # page padding untouched


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_extreme_magnitudes_bit_for_bit(fmt):
    """fp32 rows from the subnormals to the largest finite values, some of a
    block's values far below its largest: records as defined, bit for bit."""
    exps = list(range(-149, 128, 4)) + [-126, -127, 127]
    n = len(exps)
    g = torch.Generator().manual_seed(77)
    x = torch.randn((n, dims(fmt)), generator=g, dtype=torch.float64).clamp(-1.9, 1.9)
    x = x * torch.exp2(torch.tensor(exps, dtype=torch.float64))[:, None]
    x[:, ::5] *= 2.0 ** -11                     # codes at the bottom of e4m3
    x = x.float().clamp(-3.0e38, 3.0e38)
    cache = empty_cache(fmt, 128, 64)
    B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), x.cuda())
    got, want = records(cache)[:n], ENC[fmt](x).numpy()
    bad = np.argwhere(got != want)
    assert bad.size == 0, [(exps[b[0]], int(b[1]), int(got[tuple(b)]), int(want[tuple(b)])) for b in bad[:6]]


def test_write_quotients_at_ties():
    """x / s on and next to the borders between codes, for scales of every mantissa."""
    g = torch.Generator().manual_seed(78)
    n = 512
    s = (1 + torch.rand((n, 4, 1), generator=g)) * torch.exp2(torch.randint(-40, 40, (n, 4, 1), generator=g).float())
    codes = torch.arange(128, dtype=torch.uint8)[:127].view(torch.float8_e4m3fn).float()
    mids = (codes[1:] + codes[:-1]) / 2
    y = torch.cat([torch.tensor([448.0]), mids, torch.tensor([-448.0])])          # 128 values
    x = (y * s).reshape(n, 512)
    step = torch.randint(-1, 2, x.shape, generator=g)
    x = torch.where(step < 0, torch.nextafter(x, torch.zeros(())), torch.where(step > 0, torch.nextafter(x, 2 * x), x))
    cache = empty_cache(W.FMT_FP8_528, n, 64)
    B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), x.cuda())
    assert np.array_equal(records(cache)[:n], ENC[W.FMT_FP8_528](x).numpy())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("norm,style", [(True, None), (False, W.ROPE_NEOX), (False, W.ROPE_GPTJ),
                                        (True, W.ROPE_NEOX), (True, W.ROPE_GPTJ)])
@pytest.mark.parametrize("dtype", TYPES)
def test_write_norm_and_rope(fmt, norm, style, dtype):
    n, page, num = 131, 64, 256
    x = draw_rows(n, fmt, dtype, 7 + fmt)
    g = torch.Generator().manual_seed(3)
    slots = torch.randperm(num, generator=g)[:n].to(torch.int32)
    w = 1 + 0.2 * torch.randn(512, generator=g) if norm else None
    pos = torch.randint(0, W.ROPE_TABLE_ROWS, (n,), generator=g) if style is not None else None
    if pos is not None:
        pos[:2] = torch.tensor([0, W.ROPE_TABLE_ROWS - 1])
    cs = W.rope_table() if style is not None else None
    cache = empty_cache(fmt, num, page)
    cu = lambda t: None if t is None else t.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots.cuda(), x.cuda(), norm_weight=cu(w), norm_eps=1e-6, positions=cu(pos),
                      cos_sin=cu(cs), rope_style=style or 0, device_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    src = R.transform(x.float().numpy(), None if w is None else w.numpy(), 1e-6,
                      None if pos is None else pos.numpy(), None if cs is None else cs.numpy(), style or 0)
    got = R.record_values(fmt, records(cache)[slots.long().numpy()])
    mag = np.abs(src)
    if style is not None:
        ia = np.arange(32) if style == W.ROPE_NEOX else 2 * np.arange(32)
        ib = ia + (32 if style == W.ROPE_NEOX else 1)
        t = np.hypot(src[:, -64:][:, ia], src[:, -64:][:, ib]) * 2 ** 0.5
        mag[:, -64:][:, ia] = t
        mag[:, -64:][:, ib] = t
    tol = R.quant_bound(fmt, src) * (1 + 2.0 ** -10) + mag * 2.0 ** -20 + 2.0 ** -133
    err = np.abs(got - src)
    assert np.all(err <= tol), (float((err / tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 6, 300])
def test_read(fmt, dtype, n):
    page, num = 64, 1024
    g = torch.Generator(device="cuda").manual_seed(fmt)
    cache = W.make_cache(num, page, fmt, g, "cuda", page_pad=16, mag=(0, -3, 2))
    slots = torch.randint(0, num, (n,), generator=torch.Generator().manual_seed(n)).to(torch.int32)
    if n > 4:
        slots[1], slots[3], slots[4] = -1, num, slots[0]     # outside, outside, named twice
    d = dims(fmt)
    wide = torch.full((n, d + 24), 7.0, dtype=dtype, device="cuda")   # a wider row stride
    B.dsa_cache_read(cache, slots.cuda(), wide[:, :d])
    torch.cuda.synchronize()
    keep = ((slots >= 0) & (slots < num)).numpy()
    want = np.zeros((n, d))
    want[keep] = R.record_values(fmt, records(cache)[slots.numpy()[keep]])
    got = wide[:, :d].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= np.abs(want) * (HALF[dtype] + R.EPS_F32) + 2.0 ** -25)
    assert np.all(got[~keep] == 0)
    assert bool((wide[:, d:] == 7.0).all())


def test_write_wide_stride_and_offset():
    """Rows inside a wider projection (k after q), read with their stride."""
    n, fmt = 33, W.FMT_FP8_528
    big = torch.randn((n, 2048), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    rows = big[:, 1024:1536]
    cache = empty_cache(fmt, 64, 64)
    B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), rows)
    want = ENC[fmt](rows.float().cpu()).numpy()
    assert np.array_equal(records(cache)[:n], want)
    with pytest.raises(B.DsaError):      # a row that does not start on 16 bytes
        B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), big[:, 1025:1537])
    with pytest.raises(B.DsaError):      # a cache view narrower than its pages
        B.dsa_cache_write(W.PagedCache(cache.data[:, :-16], 64, fmt), torch.arange(n, dtype=torch.int32, device="cuda"), rows)
    with pytest.raises(B.DsaError):      # values that do not lie next to each other
        B.dsa_cache_write(cache, torch.arange(n, dtype=torch.int32, device="cuda"), big[:, ::4])


@pytest.mark.parametrize("fmt", FORMATS)
def test_nonfinite_rows(fmt):
    """A NaN makes its block NaN, an infinity does so or saturates; the other
    blocks and rows are those of finite rows."""
    x = draw_rows(4, fmt, torch.float32, 5, mag=False)
    size = R.block_dims(fmt)
    x[1, 3] = float("nan")
    x[2, 5] = float("-inf")
    cache = empty_cache(fmt, 64, 64)
    out = torch.empty((4, dims(fmt)), device="cuda")
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots, x.cuda())
    B.dsa_cache_read(cache, slots, out)
    o = out.cpu()
    assert bool(torch.isnan(o[1, :size]).all())
    if size == 128:
        assert bool(torch.isnan(o[2, :size]).all())
    else:
        assert float(o[2, 5]) < -1e3
    ok = torch.ones_like(o, dtype=torch.bool)
    ok[1, :size] = ok[2, :size] = False
    want = R.record_values(fmt, ENC[fmt](torch.nan_to_num(x, 0.0, 0.0, 0.0)).numpy())
    assert np.array_equal(o.double().numpy()[ok.numpy()], want.astype(np.float32).astype(np.float64)[ok.numpy()])


def test_position_outside_the_table():
    fmt, n = W.FMT_FP8_528, 4
    cs = W.rope_table(128).cuda()
    x = draw_rows(n, fmt, torch.bfloat16, 2).cuda()
    pos = torch.tensor([5, 128, -1, 127], device="cuda")
    cache = empty_cache(fmt, 64, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots, x, positions=pos, cos_sin=cs, device_status=status)
    assert int(status) == -1
    r = records(cache)
    assert np.all(r[1:3] == 0xA5) and not np.all(r[0] == 0xA5) and not np.all(r[3] == 0xA5)
    B.dsa_cache_write(cache, slots, x, positions=pos, cos_sin=cs)      # without the word: the same rows
    assert np.all(records(cache)[1:3] == 0xA5)


def test_slots_past_2_to_31_bytes():
    """Byte offsets past 32 bits: a cache of more than 4 GiB."""
    fmt, page = W.FMT_V32_656, 64
    num = ((5 << 30) // (656 * page) + 1) * page
    cache = W.PagedCache(torch.zeros((num // page, page * 656), dtype=torch.uint8, device="cuda"), page, fmt)
    x = draw_rows(3, fmt, torch.bfloat16, 9).cuda()
    slots = torch.tensor([num - 1, 0, num // 2], dtype=torch.int32, device="cuda")
    B.dsa_cache_write(cache, slots, x)
    out = torch.empty((3, 576), device="cuda")
    B.dsa_cache_read(cache, slots, out)
    want = R.record_values(fmt, ENC[fmt](x.float().cpu()).numpy())
    assert np.array_equal(out.cpu().double().numpy(), want.astype(np.float32).astype(np.float64))


def test_graph_and_other_stream():
    fmt, n = W.FMT_FP8_528_UE8M0, 40
    cache = empty_cache(fmt, 64, 64)
    x = draw_rows(n, fmt, torch.bfloat16, 4).cuda()
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    out = torch.empty((n, 512), dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        B.dsa_cache_write(cache, slots, x)
        B.dsa_cache_read(cache, slots, out)
    torch.cuda.synchronize()
    first = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dsa_cache_write(cache, slots, x)
        B.dsa_cache_read(cache, slots, out)
    x.copy_(2 * x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.float(), 2 * first.float())     # powers of two scale exactly


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_NVFP4_288, W.FMT_FP8_528_UE8M0, W.FMT_MODEL1_584])
def test_decode_reads_what_was_written(fmt):
    """Keys written by dsa_cache_write, then a decode over them against the oracle."""
    w = W.make_workload(T=6, H=64, seed=31, sink=True, device="cuda",
                        swa=dict(width=128, lens=(1, 128), fmt=fmt, page=64, slots=1024))
    x = torch.randn((1024, 512), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16).cuda()
    w.swa_cache.data.zero_()
    B.dsa_cache_write(w.swa_cache, torch.arange(1024, dtype=torch.int32, device="cuda"), x)
    dec = B.Decoder(w)
    out, lse = dec(w)
    kept, chk = dec.selection()
    torch.cuda.synchronize()
    compare(out, lse, kept, chk, oracle_ref(w), what=f"written fmt{fmt}")


def test_binding_refuses_what_pointers_cannot_tell():
    fmt, n = W.FMT_FP8_528, 8
    cache = empty_cache(fmt, 64, 64)
    ok = dict(slots=torch.arange(n, dtype=torch.int32, device="cuda"), rows=torch.zeros((n, 512), device="cuda"))
    w, pos, cs = torch.ones(512, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda"), W.rope_table(16, "cuda")
    B.dsa_cache_write(cache, **ok, norm_weight=w, positions=pos, cos_sin=cs)
    bad = [dict(slots=ok["slots"].long()), dict(slots=ok["slots"][::2]), dict(slots=ok["slots"].view(2, 4)),
           dict(slots=ok["slots"].cpu()), dict(slots=None), dict(rows=ok["rows"].double()), dict(rows=ok["rows"][:, :511]),
           dict(rows=ok["rows"][1:]), dict(rows=ok["rows"].t()), dict(rows=ok["rows"].cpu()), dict(norm_weight=w[:511]),
           dict(norm_weight=w.to(torch.bfloat16)), dict(positions=pos.int(), cos_sin=cs), dict(positions=pos[1:], cos_sin=cs),
           dict(positions=pos, cos_sin=cs[:, :32]), dict(positions=pos, cos_sin=cs.double()), dict(positions=pos),
           dict(device_status=pos), dict(device_status=torch.zeros(1, dtype=torch.int32))]
    before = cache.data.clone()
    for kw in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_cache_write(cache, **dict(ok, **kw))
        assert e.value.status == -1
    for c in (W.PagedCache(cache.data.to(torch.int8), 64, fmt), W.PagedCache(cache.data.t(), 64, fmt),
              W.PagedCache(cache.data.cpu(), 64, fmt), W.PagedCache(cache.data.view(-1), 64, fmt)):
        with pytest.raises(B.DsaError):
            B.dsa_cache_read(c, ok["slots"], ok["rows"])
    assert torch.equal(cache.data, before)
    st = torch.cuda.Stream()
    B.dsa_cache_read(cache, ok["slots"], ok["rows"], stream=st)          # a stream, or its raw handle
    B.dsa_cache_read(cache, ok["slots"], ok["rows"], stream=st.cuda_stream)
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_rows(fmt):
    """A step without new keys: every argument empty, the table there."""
    cache = empty_cache(fmt, 64, 64)
    none = dict(slots=torch.empty(0, dtype=torch.int32, device="cuda"), rows=torch.empty((0, dims(fmt)), device="cuda"))
    w, cs = torch.ones(512, device="cuda"), W.rope_table(16, "cuda")
    B.dsa_cache_write(cache, **none)
    B.dsa_cache_write(cache, **none, norm_weight=w, norm_eps=1e-6, cos_sin=cs,
                      positions=torch.empty(0, dtype=torch.int64, device="cuda"))
    B.dsa_cache_read(cache, **none)
    torch.cuda.synchronize()
    assert bool((cache.data == 0xA5).all())
