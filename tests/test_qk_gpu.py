"""dsa_qk_norm on the GPU against the formulas in 64 bits, and against
dsa_cache_write for the keys (the same records bit for bit).

Tolerance of the queries. In fp32 the sum of 512 squares takes 4 fused adds, a
few sums and 5 exchanges: 2^-20.5 of it at most, half of that in its root;
the reciprocal root is good to 2^-22, the two products to 2^-24 each: together
below 2^-20 of a value. The rotation's products and sum add 2^-23 of |a c| +
|b s|. The result is rounded to bf16: half a step, 2^-8 of it."""
import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import _cache_ref as R

pytestmark = pytest.mark.gpu
FORMATS = list(W.RECORD_BYTES)
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def empty(fmt, n, page=16):
    pages = -(-n // page)
    return W.PagedCache(torch.full((pages, page * W.RECORD_BYTES[fmt]), 0xA5, dtype=torch.uint8, device="cuda"), page, fmt)


def reference(q, weight, eps, pos, cs, style):
    """-> rows in 64 bits, and the magnitudes that their rounding errors go by."""
    T, H, d = q.shape
    x = q.double().cpu().numpy().reshape(T * H, d).copy()
    if weight is not None:
        w = weight.double().cpu().numpy()
        w = np.tile(w if w.ndim == 2 else w[None], (T if w.ndim == 2 else T * H, 1))
        v = x[:, :512]
        m = np.maximum(np.abs(v).max(1, keepdims=True), 1e-300)     # (squares of large and small rows)
        rms = m * np.sqrt(((v / m) ** 2).mean(1, keepdims=True) + eps / m / m)
        x[:, :512] = v / rms * w
    mag = np.abs(x).copy()
    if pos is not None:
        p = np.repeat(pos.cpu().numpy(), H)
        t = cs.cpu().numpy().astype(np.float64)
        mag = R.transform(mag, positions=p, cos_sin=np.concatenate([np.abs(t[:, :32]), np.abs(t[:, 32:])], 1), style=style)
        alt = R.transform(np.abs(x), positions=p, cos_sin=np.concatenate([np.abs(t[:, :32]), -np.abs(t[:, 32:])], 1), style=style)
        mag = np.maximum(np.abs(mag), np.abs(alt))                  # |a c| + |b s| is one of the two
        x = R.transform(x, positions=p, cos_sin=t, style=style)
    return x.reshape(T, H, d), mag.reshape(T, H, d)


def check(out, want, mag):
    got = out.double().cpu().numpy()
    tol = np.abs(want) * 2.0 ** -8 + mag * 2.0 ** -18 + 2.0 ** -133
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol), float((np.abs(got - want) / tol).max())


def make(T, H, fmt, type, seed, norm=True, rope=W.ROPE_NEOX, per_head=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = 576 if fmt == W.FMT_V32_656 else 512
    q = torch.randn((T, H, d), generator=g, device="cuda").to(type)
    k = (2 * torch.randn((T, d), generator=g, device="cuda")).to(type)
    qw = 1 + 0.2 * torch.randn((H, 512) if per_head else (512,), generator=g, device="cuda") if norm else None
    kw = 1 + 0.2 * torch.randn((512,), generator=g, device="cuda") if norm else None
    pos = cs = None
    if rope is not None:
        cs, pos = W.rope_table(4096, "cuda"), torch.randint(0, 4096, (T,), generator=g, device="cuda")
    slots = torch.randperm(T + 5, generator=g, device="cuda")[:T].to(torch.int32)
    if T > 3:
        slots[2] = -1
    return q, k, qw, kw, slots, dict(eps=1e-6, positions=pos, cos_sin=cs, rope_style=rope or 0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("norm,rope", [(True, W.ROPE_NEOX), (True, W.ROPE_GPTJ), (False, W.ROPE_NEOX), (False, W.ROPE_GPTJ),
                                       (True, None), (False, None)])
def test_against_the_formula(fmt, type, norm, rope):
    T, H = 9, 20
    q, k, qw, kw, slots, kw_args = make(T, H, fmt, type, fmt, norm, rope)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cache, same = empty(fmt, T + 5), empty(fmt, T + 5)
    B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, **kw_args)
    B.dsa_cache_write(same, slots, k, kw, 1e-6, kw_args["positions"], kw_args["cos_sin"], kw_args["rope_style"])
    torch.cuda.synchronize()
    check(out, *reference(q, qw, 1e-6, kw_args["positions"], kw_args["cos_sin"], kw_args["rope_style"]))
    assert torch.equal(cache.data, same.data)


@pytest.mark.parametrize("T,H", [(1, 1), (1, 128), (2, 3), (700, 16), (40, 130), (3000, 1)])
@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_V32_656])
def test_sizes(T, H, fmt):
    """Fewer rows than warps, more, and more keys than query blocks."""
    q, k, qw, kw, slots, args = make(T, H, fmt, torch.bfloat16, T)
    out = torch.empty_like(q)
    cache, same = empty(fmt, T + 5), empty(fmt, T + 5)
    B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, **args)
    B.dsa_cache_write(same, slots, k, kw, 1e-6, args["positions"], args["cos_sin"])
    torch.cuda.synchronize()
    check(out, *reference(q, qw, 1e-6, args["positions"], args["cos_sin"], 0))
    assert torch.equal(cache.data, same.data)


def test_queries_alone_in_place_and_strided():
    q, _, qw, _, _, args = make(6, 16, W.FMT_FP8_528, torch.bfloat16, 3)
    want = torch.empty_like(q)
    B.dsa_qk_norm(q, want, qw, **args)
    torch.cuda.synchronize()
    check(want, *reference(q, qw, 1e-6, args["positions"], args["cos_sin"], 0))
    for off, wide in ((512, 1024), (8, 536)):        # 32- and 16-byte aligned rows
        src = torch.full((6, 16, wide), 3.0, dtype=torch.bfloat16, device="cuda")
        src[:, :, off:off + 512] = q
        dst = torch.full((6, 16, wide), 5.0, dtype=torch.bfloat16, device="cuda")
        B.dsa_qk_norm(src[:, :, off:off + 512], dst[:, :, off:off + 512], qw, **args)
        torch.cuda.synchronize()
        assert torch.equal(dst[:, :, off:off + 512], want)
        dst[:, :, off:off + 512] = 5
        assert bool((dst == 5).all())
        B.dsa_qk_norm(src[:, :, off:off + 512], src[:, :, off:off + 512], qw, **args)
        torch.cuda.synchronize()
        assert torch.equal(src[:, :, off:off + 512], want)
    heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)      # a head stride above the token stride
    with pytest.raises(B.DsaError):
        B.dsa_qk_norm(heads_first, want, qw, **args)


def test_weights_per_head():
    q, _, qw, _, _, args = make(5, 20, W.FMT_FP8_528, torch.float32, 4, per_head=True)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    B.dsa_qk_norm(q, out, qw, **args)
    torch.cuda.synchronize()
    check(out, *reference(q, qw, 1e-6, args["positions"], args["cos_sin"], 0))


@pytest.mark.parametrize("log2", [-120, -80, -40, 40, 70, 115])
def test_magnitudes(log2):
    """Rows whose squares leave fp32's range."""
    q, _, qw, _, _, args = make(4, 16, W.FMT_FP8_528, torch.float32, 5)
    q = q * 2.0 ** log2
    q[1] *= 2.0 ** (-10 if log2 > 0 else 10)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device="cuda")
    args["eps"] = 0.0
    B.dsa_qk_norm(q, out, qw, **args)
    torch.cuda.synchronize()
    check(out, *reference(q, qw, 0.0, args["positions"], args["cos_sin"], 0))


def test_zeros_infinities_and_nan_stay_in_their_rows():
    q, _, qw, _, _, args = make(4, 16, W.FMT_FP8_528, torch.bfloat16, 6)
    q[0, 3] = 0
    clean = torch.empty_like(q)
    B.dsa_qk_norm(q, clean, qw, **args)
    bad = q.clone()
    bad[1, 5, 100], bad[2, 6, 500] = float("nan"), float("inf")
    out = torch.empty_like(q)
    B.dsa_qk_norm(bad, out, qw, **args)
    torch.cuda.synchronize()
    assert bool((clean[0, 3] == 0).all()) and bool(torch.isnan(out[1, 5]).all()) and bool(torch.isnan(out[2, 6]).any())
    ok = torch.ones((4, 16), dtype=torch.bool, device="cuda")
    ok[1, 5] = ok[2, 6] = False
    assert torch.equal(out[ok], clean[ok])


def test_a_position_outside_the_table_writes_nothing_of_the_token():
    q, k, qw, kw, slots, args = make(6, 16, W.FMT_FP8_528, torch.bfloat16, 7)
    args["positions"][1], args["positions"][4] = 4096, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cache = empty(W.FMT_FP8_528, 11)
    B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, device_status=status, **args)
    torch.cuda.synchronize()
    assert int(status) == -1
    rec = cache.data.view(-1, 528)
    for t in range(6):
        outside = t in (1, 4)
        assert bool((out[t] == 7).all()) == outside
        if int(slots[t]) >= 0:
            assert bool((rec[int(slots[t])] == 0xA5).all()) == outside


def test_captured():
    q, k, qw, kw, slots, args = make(33, 64, W.FMT_MODEL1_584, torch.bfloat16, 8)
    out = torch.empty_like(q)
    cache = empty(W.FMT_MODEL1_584, 38)
    B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, **args)
    torch.cuda.synchronize()
    want, rec = out.clone(), cache.data.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.dsa_qk_norm(q, out, qw, k, kw, cache, slots, **args)
    out.zero_()
    cache.data.fill_(0xA5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.data, rec)


def test_binding_refuses_what_pointers_cannot_tell():
    q, k, qw, kw, slots, args = make(6, 16, W.FMT_FP8_528, torch.bfloat16, 9)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cache = empty(W.FMT_FP8_528, 11)
    ok = dict(q=q, out=out, q_weight=qw, keys=k, key_weight=kw, cache=cache, slots=slots, **args)
    bad = [dict(q=q.double()), dict(q=q[:, :, :500]), dict(q=q[0]), dict(q=q.cpu()), dict(out=out.float()), dict(out=out[:5]),
           dict(q_weight=qw[:500]), dict(q_weight=qw.repeat(3, 1)), dict(q_weight=qw.double()), dict(keys=None), dict(keys=k[:5]),
           dict(keys=k.float()), dict(key_weight=kw[:100]), dict(slots=None), dict(slots=slots.long()), dict(slots=slots[:4]),
           dict(cache=None), dict(positions=None), dict(positions=args["positions"].int()), dict(cos_sin=None),
           dict(cos_sin=args["cos_sin"][:, :60]), dict(rope_style=3), dict(eps=-1.0), dict(eps=float("nan")),
           dict(device_status=slots), dict(cache=empty(W.FMT_V32_656, 11)), dict(q=torch.zeros((6, 16, 576), dtype=q.dtype, device="cuda"))]
    for kw_ in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_qk_norm(**dict(ok, **kw_))
        assert e.value.status == -1, kw_
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((cache.data == 0xA5).all())
