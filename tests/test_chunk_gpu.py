"""dsa_chunk_run on the GPU against the formulas in 64 bits.

Tolerances: those of the shared-prefix attention, whose kernels these are
(test_prefix_gpu.py derives them): scores off by delta <= (2^-10 + 2^-13) A +
2^-17, A the sum of the products' magnitudes; lse by delta and 2^-18 of itself;
the output by weights off by e^{+-2 delta}, 2^-11 of a weight, 2^-11 of a value
and bf16's half step 2^-8."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests._serve_ref import Batch

pytestmark = pytest.mark.gpu
FORMATS = list(W.RECORD_BYTES)
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def attention(c, num_sms=0):
    return B.ChunkAttention(c.T, c.B, c.H, c.width, "cuda", c.d, num_sms)


def call(c, attn, **kw):
    return attn(c.q, c.cache, c.slots, c.lengths, c.starts, c.scale, c.window, c.sink, c.pos, c.cs, c.style, c.tail_out,
                c.tail_lse, **kw)


def run(c, num_sms=0, attn=None):
    attn = attn or attention(c, num_sms)
    attn.out.fill_(7.0)
    attn.lse.fill_(7.0)
    out, lse = call(c, attn)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == 0
    return out, lse, attn


def reference(c):
    """-> out, lse, their largest errors, and the tokens that belong to a sequence."""
    out = torch.zeros((c.T, c.H, 512), dtype=torch.float64, device="cuda")
    lse = torch.full((c.T, c.H), -INF, dtype=torch.float64, device="cuda")
    mag, delta = torch.zeros_like(out), torch.zeros_like(lse)
    own = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for b, t, at, k, x, mass in c.scores():
        n = x.shape[0]
        own[t:t + n] = True
        if n == 0 or len(at) == 0:
            continue
        l = torch.logsumexp(x, 2)
        w = torch.where(torch.isfinite(l)[..., None], (x - l[..., None]).exp(), torch.zeros_like(x))
        lse[t:t + n], out[t:t + n], mag[t:t + n] = l, w @ k[:, :512], w @ k[:, :512].abs()
        delta[t:t + n] = mass.amax(2)
    delta = (2.0 ** -10 + 2.0 ** -13) * delta + 2.0 ** -17
    both = lse
    if c.tail_lse is not None:
        tl, to = c.tail_lse.double(), c.tail_out.double().nan_to_num()
        both = torch.logaddexp(lse, tl)
    den = both if c.sink is None else torch.logaddexp(both, c.sink.double())

    def weight(l):
        return torch.where(torch.isfinite(l), (l - den).exp(), torch.zeros_like(l))[..., None]

    out, mag = weight(lse) * out, weight(lse) * mag
    if c.tail_lse is not None:
        out, mag = out + weight(tl) * to, mag + weight(tl) * to.abs()
    tol = torch.expm1(2 * delta)[..., None] * (mag + out.abs()) + 2.0 ** -10 * mag
    tol = tol + (out.abs() + tol) * 2.0 ** -8 + 2.0 ** -126
    ltol = delta + torch.where(torch.isfinite(both), both.abs(), torch.zeros_like(both)) * 2.0 ** -18
    return out, both, tol, ltol, own


def check(c, out, lse):
    r_out, r_lse, tol, ltol, own = reference(c)
    assert bool((out[~own] == 7).all()) and bool((lse[~own] == 7).all())     # left as they were
    out, lse, r_out, r_lse, tol, ltol = (x[own] for x in (out.double(), lse.double(), r_out, r_lse, tol, ltol))
    fin = torch.isfinite(r_lse)
    assert torch.equal(torch.isfinite(lse), fin) and bool((lse[~fin] == -INF).all())
    assert bool((out[~fin] == 0).all())
    bad = (lse[fin] - r_lse[fin]).abs() > ltol[fin]
    assert not bool(bad.any()), float(((lse[fin] - r_lse[fin]).abs() / ltol[fin]).max())
    bad = (out - r_out).abs() > tol
    assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), float(((out - r_out).abs() / tol).max()))
    if float(r_out.norm()) > 0:   # roundings of either sign
        assert float((out - r_out).norm() / r_out.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,H", [([(1, 1)], 1), ([(1, 128)], 64), ([(7, 129), (1, 3)], 20), ([(16, 300), (1, 257), (40, 40)], 16)])
def test_plain(fmt, sizes, H):
    c = Batch(sizes, H, fmt, seed=fmt)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 100, 128])
def test_everything_on(fmt, window):
    rope = None if fmt == W.FMT_V32_656 else (W.ROPE_NEOX if window else W.ROPE_GPTJ)
    c = Batch([(33, 700), (1, 513), (0, 90), (5, 5), (90, 612)], 20, fmt, seed=5, width=720, invalid=0.1, rope=rope, sink=True,
              tail=True, window=window, page_pad=32, before=3, behind=4)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600, 2**31 - 1])
def test_windows(window):
    c = Batch([(70, 500), (1, 256), (200, 200)], 16, W.FMT_FP8_528_UE8M0, seed=window % 97, window=window)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("length", [0, -3, 1, 4, 5, 6, 127, 128, 129, 255, 256, 257, 1 << 20])
@pytest.mark.parametrize("window", [0, 3])
def test_lengths(length, window):
    """Lists shorter than the chunk leave its first tokens without keys."""
    c = Batch([(5, length), (2, 30)], 40, W.FMT_FP8_528, width=300, seed=6, window=window, sink=True)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("sms", [2, 4, 8, 12, 28, 152])
@pytest.mark.parametrize("tail", [False, True])
def test_splits(sms, tail):
    """Row tiles whole in a pair, shared by two, cut into many."""
    c = Batch([(9, 1100), (1, 40), (30, 800), (1, 1300)], 32, W.FMT_NVFP4_288, seed=sms, sink=True, tail=tail)
    out, lse, attn = run(c, sms)
    assert attn.plan.pairs == min(sms // 2, attn.plan.pairs)
    check(c, out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("sms", [2, 6])
def test_whole_tiles_with_rows_that_end_inside_a_warp(fmt, tail, sms):
    """Several tiles to a pair, whole and shared, whose last rows are not 32."""
    c = Batch([(17, 300), (1, 40), (20, 500), (9, 9)], 20, fmt, seed=sms, sink=True, tail=tail, window=0 if sms == 2 else 150)
    check(c, *run(c, sms)[:2])


def test_no_slot_kept():
    c = Batch([(3, 300), (4, 200)], 16, W.FMT_FP8_528, seed=6, tail=True)
    c.slots[0] = -1
    check(c, *run(c)[:2])
    c = Batch([(3, 600)], 16, W.FMT_FP8_528, seed=7)
    c.slots[0, :300] = -1
    c.slots[0, -30:] = c.cache.num_slots
    check(c, *run(c, 2)[:2])


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_MODEL1_584, W.FMT_V32_656])
@pytest.mark.parametrize("mag,q_log2", [((-20,), 20), ((16,), -16), ((0, 0, 0, 12, -9), -10)])
def test_magnitudes(fmt, mag, q_log2):
    c = Batch([(20, 400), (3, 70)], 32, fmt, seed=11, mag=mag, q_log2=q_log2, window=200)
    check(c, *run(c)[:2])


def test_many_sequences():
    """More sequences than the blocks scan at a time, some of them empty."""
    sizes = [(i % 3, 1 + (37 * i) % 200) for i in range(700)]
    c = Batch(sizes, 8, W.FMT_NVFP4_288, seed=8, width=200, window=64, sink=True, num_slots=8192)
    check(c, *run(c)[:2])


def test_many_row_tiles():
    c = Batch([(150, 400), (1, 60), (130, 130)], 128, W.FMT_FP8_528_UE8M0, seed=14, rope=W.ROPE_GPTJ, sink=True, tail=True)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("H", [1, 7, 200, 300])
def test_any_head_count(H):
    """Row tiles that begin and end inside a token's heads."""
    c = Batch([(5, 300), (1, 40), (9, 150)], H, W.FMT_FP8_528_UE8M0, seed=H, sink=True, window=100)
    for sms in (4, 0):
        check(c, *run(c, sms)[:2])


def test_outputs_on_16_byte_boundaries():
    c = Batch([(30, 300), (9, 150)], 64, W.FMT_NVFP4_288, seed=3, sink=True)
    for tail in (False, True):
        if tail:
            c.tail_out, c.tail_lse = 0.1 * torch.ones((c.T, 64, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((c.T, 64), device="cuda")
        for sms in (2, 0):
            attn = attention(c, sms)
            room = torch.full((c.T * 64 * 512 + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
            attn.out = room[8:-8].view(c.T, 64, 512)
            assert attn.out.data_ptr() % 32 == 16
            check(c, *run(c, attn=attn)[:2])
            assert bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())


@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_negative_and_zero_scale(scale):
    c = Batch([(20, 300)], 16, W.FMT_NVFP4_288, seed=33)
    c.scale = scale
    check(c, *run(c)[:2])


def test_no_tokens_in_any_sequence():
    c = Batch([(0, 30), (0, 0)], 16, W.FMT_FP8_528, seed=4, behind=5)
    check(c, *run(c)[:2])


@pytest.mark.parametrize("window", [0, 50])
def test_what_the_workspace_held_does_not_count(window):
    """Images of keys that no record fills are zeros wherever a product takes them."""
    c = Batch([(3, 300), (1, 17), (20, 450), (1, 1)], 20, W.FMT_FP8_528, seed=2, invalid=0.1, window=window)
    attn = attention(c)
    for byte in (0xFF, 0x7C):   # NaN, and large numbers and infinities
        attn.workspace.fill_(byte)
        check(c, *run(c, attn=attn)[:2])


def test_long_list_of_few_tokens():
    c = Batch([(2, 70000)], 16, W.FMT_NVFP4_288, seed=13, num_slots=4096)
    check(c, *run(c)[:2])


def test_strides():
    c = Batch([(4, 200), (6, 150)], 16, W.FMT_FP8_528, seed=15)
    wide = torch.zeros((c.T, 16, 1024), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 512:] = c.q
    c.q = wide[:, :, 512:]
    lists = torch.full((2, 333), 5, dtype=torch.int32, device="cuda")
    lists[:, :200] = c.slots
    c.slots = lists[:, :200]
    check(c, *run(c)[:2])


def test_one_head_of_one_token_as_a_decode_step():
    """Single tokens give what the decode gives for the same lists."""
    w = W.make_workload(T=6, H=64, seed=41, sink=True, rope=True, rope_style=W.ROPE_NEOX, device="cuda",
                        swa=dict(width=128, lens=(1, 128), fmt=W.FMT_FP8_528, page=64, slots=2048))
    dec = B.Decoder(w)
    o1, l1 = dec(w)
    attn = B.ChunkAttention(6, 6, 64, 128, "cuda")
    o2, l2 = attn(w.q, w.swa_cache, w.swa.ids, w.swa.lens, torch.arange(7, dtype=torch.int32, device="cuda"), w.scale, 0, w.sink,
                  w.positions, w.cos_sin)
    torch.cuda.synchronize()
    assert float((l1 - l2).abs().max()) <= 1e-3 and float((o1.float() - o2.float()).abs().max()) <= 2e-2


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("what", ["scale", "value"])
def test_nan_key_reaches_the_rows_that_see_it(fmt, what):
    """and no other row: not the tokens before it, not those whose window it left."""
    c = Batch([(40, 300)], 16, fmt, seed=17, window=20)
    c.slots[c.slots == 0] = -1
    c.slots[0, 270] = 0                      # the position of token 10
    want = [t.clone() for t in run(c)[:2]]
    rec = c.cache.data[0, :c.cache.record_bytes]
    at = {W.FMT_FP8_528: (512, 5), W.FMT_FP8_528_UE8M0: (520, 5), W.FMT_NVFP4_288: (260, 260), W.FMT_MODEL1_584: (578, 450),
          W.FMT_V32_656: (512, 530)}[fmt][what == "value"]
    if what == "scale" and fmt in (W.FMT_FP8_528, W.FMT_V32_656):
        rec[at:at + 4].view(torch.float32).fill_(float("inf"))
    elif at in (450, 530):
        rec[at:at + 2].view(torch.bfloat16).fill_(float("nan"))
    else:
        rec[at] = 0x7F if what == "value" or fmt == W.FMT_NVFP4_288 else 0xFF
    out, lse, _ = run(c)
    sees = torch.zeros(40, dtype=torch.bool, device="cuda")
    sees[10:30] = True
    assert bool(torch.isnan(lse[sees]).all()) and bool(torch.isnan(out[sees]).all())
    assert bool(torch.isfinite(lse[~sees]).all())
    # (the group's exponents may differ, and with them a rounding)
    assert float((lse[~sees] - want[1][~sees]).abs().max()) <= 1e-4
    assert float((out[~sees].float() - want[0][~sees].float()).abs().max()) <= 2e-2


def test_starts_out_of_order_leave_everything():
    c = Batch([(3, 300), (4, 200)], 16, W.FMT_FP8_528, seed=18)
    attn = attention(c)
    for bad in ([0, 5, 4], [-1, 3, 7], [0, 3, 8], [2**31 - 1, 3, 7]):
        attn.out.fill_(7.0)
        attn.lse.fill_(7.0)
        attn(c.q, c.cache, c.slots, c.lengths, torch.tensor(bad, dtype=torch.int32, device="cuda"), c.scale)
        assert B.dsa_decode_read_status(attn.workspace) == -1
        assert bool((attn.out == 7).all()) and bool((attn.lse == 7).all())
    check(c, *run(c, attn=attn)[:2])


def test_position_outside_the_table_sets_the_status():
    c = Batch([(2, 200)], 16, W.FMT_FP8_528, seed=18, rope=W.ROPE_NEOX)
    c.pos[1] = 4096
    attn = attention(c)
    call(c, attn)
    assert B.dsa_decode_read_status(attn.workspace) == -1
    c.pos[1] = 0
    check(c, *run(c, attn=attn)[:2])


def test_in_place_tail():
    c = Batch([(9, 500), (1, 700)], 64, W.FMT_FP8_528, seed=16, sink=True, tail=True)
    out, lse, attn = run(c)
    o, l = c.tail_out.clone(), c.tail_lse.clone()
    B.dsa_chunk_run(attn.plan, attn.workspace, c.q, c.cache, c.slots, c.lengths, c.starts, 0, c.sink, None, None, 0, c.scale, o, l,
                    o, l)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l.view(torch.int32), lse.view(torch.int32))


def test_reproducible_and_captured():
    c = Batch([(60, 900), (1, 1500), (20, 333)], 64, W.FMT_FP8_528, seed=19, rope=W.ROPE_NEOX, sink=True, tail=True)
    out, lse, attn = run(c)
    want = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, attn)
    for _ in range(3):
        attn.out.fill_(7.0)
        attn.lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(attn.out.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(attn.lse.view(torch.int32), want[1].view(torch.int32))
    # lengths and starts that change between replays are read by the kernels
    c.sizes = [(10, 70), (61, 1400), (10, 10)]
    c.lengths.copy_(torch.tensor([70, 1400, 10]))
    c.starts.copy_(torch.tensor([0, 10, 71, 81]))
    g.replay()
    torch.cuda.synchronize()
    check(c, attn.out, attn.lse)


def test_two_streams_with_their_own_workspaces():
    cs = [Batch([(30, 900), (9, 1500)], 64, W.FMT_FP8_528, seed=20 + i, sink=True) for i in range(2)]
    want = [tuple(t.clone() for t in run(c)[:2]) for c in cs]
    attn = [attention(c) for c in cs]
    st = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, a, s in zip(cs, attn, st):
            call(c, a, stream=s)
    torch.cuda.synchronize()
    for w, a in zip(want, attn):
        assert torch.equal(a.out, w[0]) and torch.equal(a.lse, w[1])


def test_short_wait_budget_reports_a_timeout(monkeypatch):
    c = Batch([(40, 1000)], 64, W.FMT_FP8_528, seed=50)
    monkeypatch.setenv("DSA_DECODE_WAIT_BUDGET", "1")
    attn = attention(c)
    monkeypatch.delenv("DSA_DECODE_WAIT_BUDGET")
    call(c, attn)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == -6
    check(c, *run(c)[:2])


def test_binding_refuses_what_pointers_cannot_tell():
    c = Batch([(2, 300), (3, 100)], 16, W.FMT_FP8_528, seed=60, rope=W.ROPE_NEOX, sink=True, tail=True)
    out, _, attn = run(c)
    want = out.clone()
    ok = dict(plan=attn.plan, workspace=attn.workspace, q=c.q, cache=c.cache, slots=c.slots, lengths=c.lengths, starts=c.starts,
              window=0, sink=c.sink, positions=c.pos, cos_sin=c.cs, rope_style=0, scale=c.scale, tail_out=c.tail_out,
              tail_lse=c.tail_lse, out=attn.out, lse=attn.lse)
    bad = [dict(q=c.q.float()), dict(q=c.q[:1]), dict(q=c.q.cpu()), dict(slots=c.slots[:, :299]), dict(slots=c.slots[:1]),
           dict(slots=c.slots.long()), dict(slots=c.slots.t()), dict(lengths=c.lengths[:1]), dict(lengths=c.lengths.long()),
           dict(starts=c.starts[:2]), dict(starts=c.starts.long()), dict(window=-1), dict(window=2**31), dict(sink=c.sink[:8]),
           dict(positions=None), dict(cos_sin=c.cs[:, :60]), dict(tail_out=None), dict(tail_lse=c.tail_lse[:1]),
           dict(out=attn.out.float()), dict(lse=attn.lse.t()), dict(scale=float("nan")), dict(rope_style=2)]
    for kw in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_chunk_run(**dict(ok, **kw))
        assert e.value.status == -1, kw
    with pytest.raises(B.DsaError) as e:
        B.dsa_chunk_run(**dict(ok, workspace=attn.workspace[:1024]))
    assert e.value.status == -4
    torch.cuda.synchronize()
    assert torch.equal(attn.out, want)
