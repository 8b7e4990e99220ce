"""dsa_prefix_run on the GPU against the formulas in 64 bits.

Tolerances. A key's value is off by at most 2^-11 relative in the f16 tile
(fp32 product, one rounding), a rotated query value too (2^-11; without a
table queries are exact), the tensor core's fp32 sum by less than 2^-13 of
the sum of magnitudes: with A = scale * sum_i |q_i k_i| the scores are off
by delta <= (2^-10 + 2^-13) A + 2^-17, where the last term covers the fp32
work on the scores (|y| < 2^6 in units of 2^-24, a few roundings). lse is
off by at most delta (and 2^-18 relative for its own sum and log). The
output is a mean of values with weights off by e^{+-2 delta}, by 2^-11
(P in f16) and values off by 2^-11, then rounded to bf16 (2^-8).
"""
import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import _cache_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


class Case:
    def __init__(self, T, H, width, fmt, *, seed=0, page=64, length=None, invalid=0.0, rope=None,
                 sink=False, tail=False, mag=(0,), q_log2=0, num_slots=None, page_pad=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.width, self.fmt = T, H, width, fmt
        self.d = 576 if fmt == W.FMT_V32_656 else 512
        num_slots = num_slots or -(-(width + 64) // page) * page
        self.cache = W.make_cache(num_slots, page, fmt, g, "cuda", page_pad, mag=mag)
        if width <= num_slots:
            self.slots = torch.randperm(num_slots, generator=g, device="cuda")[:width].to(torch.int32)
        else:
            self.slots = torch.randint(0, num_slots, (width,), generator=g, device="cuda").to(torch.int32)
        if invalid:
            drop = torch.rand((width,), generator=g, device="cuda")
            self.slots[drop < invalid] = -1
            self.slots[drop > 1 - invalid / 2] = num_slots
        self.length = torch.tensor([width if length is None else length], dtype=torch.int32, device="cuda")
        self.q = (torch.randn((T, H, self.d), generator=g, device="cuda") * 2.0 ** q_log2).to(torch.bfloat16)
        self.scale = self.d ** -0.5
        self.sink = torch.randn((H,), generator=g, device="cuda") if sink else None
        self.tail_out = self.tail_lse = None
        if tail:
            self.tail_out = (0.3 * torch.randn((T, H, 512), generator=g, device="cuda")).to(torch.bfloat16)
            self.tail_lse = 3 + 2 * torch.randn((T, H), generator=g, device="cuda")
            if T * H > 2:
                self.tail_lse.view(-1)[1] = -float("inf")     # a token without a list of its own
                self.tail_out.view(-1, 512)[1] = float("nan")
        self.style = rope or 0
        self.pos = self.cs = None
        if rope is not None:
            self.cs = W.rope_table(4096, "cuda")
            self.pos = torch.randint(0, 4096, (T,), generator=g, device="cuda")

    def run(self, num_sms=0, attn=None):
        attn = attn or B.PrefixAttention(self.T, self.H, self.width, "cuda", self.d, num_sms)
        attn.out.fill_(float("nan"))
        attn.lse.fill_(float("nan"))
        out, lse = attn(self.q, self.cache, self.slots, self.length, self.scale, self.sink, self.pos, self.cs,
                        self.style, self.tail_out, self.tail_lse)
        torch.cuda.synchronize()
        assert B.dsa_decode_read_status(attn.workspace) == 0
        return out, lse, attn

    def reference(self):
        """-> out, lse, and the largest errors that the roundings allow of both."""
        rb = self.cache.record_bytes
        rec = self.cache.data[:, :self.cache.page_size * rb].reshape(-1, rb).cpu().numpy()
        ids = self.slots.cpu().numpy()
        n = min(max(int(self.length), 0), self.width)
        ids = ids[:n][(ids[:n] >= 0) & (ids[:n] < len(rec))]
        k = R.record_values(self.fmt, rec[ids]) if len(ids) else np.zeros((0, self.d))
        q = self.q.double().cpu().numpy().reshape(self.T * self.H, self.d)
        if self.pos is not None:
            q = R.transform(q, positions=np.repeat(self.pos.cpu().numpy(), self.H), cos_sin=self.cs.cpu().numpy(),
                            style=self.style)
        s = self.scale * (q @ k.T)
        mass = self.scale * (np.abs(q) @ np.abs(k).T)
        delta = (2.0 ** -10 + 2.0 ** -13) * mass.max(1, initial=0.0) + 2.0 ** -17
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            m = np.where(len(ids) > 0, s.max(1, initial=-np.inf), -np.inf)
            w = np.exp(s - np.where(np.isfinite(m), m, 0)[:, None])
            z = w.sum(1)
            lse = np.where(z > 0, np.where(np.isfinite(m), m, 0) + np.log(z), -np.inf)
            v = k[:, :512]
            o = (w @ v) / np.where(z > 0, z, 1)[:, None]
            oa = (w @ np.abs(v)) / np.where(z > 0, z, 1)[:, None]
            both = lse
            if self.tail_lse is not None:
                tl = self.tail_lse.double().cpu().numpy().reshape(-1)
                to = np.nan_to_num(self.tail_out.double().cpu().numpy().reshape(-1, 512))
                both = np.logaddexp(lse, tl)
            den = both if self.sink is None else np.logaddexp(both, np.tile(self.sink.double().cpu().numpy(), self.T))
            wp = np.where(np.isfinite(lse), np.exp(lse - den), 0)[:, None]
            out, mag = wp * o, wp * oa
            if self.tail_lse is not None:
                wt = np.where(np.isfinite(tl), np.exp(tl - den), 0)[:, None]
                out, mag = out + wt * to, mag + wt * np.abs(to)
        tol = np.expm1(2 * delta)[:, None] * (mag + np.abs(out)) + 2.0 ** -10 * mag
        tol = tol + (np.abs(out) + tol) * 2.0 ** -8 + 2.0 ** -126
        ltol = delta + np.where(np.isfinite(both), np.abs(both), 0) * 2.0 ** -18
        return out, both, tol, ltol

    def check(self, out, lse):
        r_out, r_lse, tol, ltol = self.reference()
        o = out.double().cpu().numpy().reshape(r_out.shape)
        l = lse.double().cpu().numpy().reshape(r_lse.shape)
        fin = np.isfinite(r_lse)
        assert np.array_equal(np.isfinite(l), fin) and np.all(l[~fin] == -np.inf)
        dl = np.abs(l[fin] - r_lse[fin])
        assert np.all(dl <= ltol[fin]), float((dl / ltol[fin]).max())
        assert np.all(o[~fin] == 0)
        bad = np.abs(o - r_out) > tol
        assert not bad.any(), (np.argwhere(bad)[:4], float((np.abs(o - r_out) / tol).max()))
        n = np.linalg.norm(r_out)
        if n > 0:   # roundings of either sign: the bf16 half step bounds them together
            rel = np.linalg.norm(o - r_out) / n
            assert rel <= 2.0 ** -8, rel
            return rel
        return 0.0


FORMATS = list(W.RECORD_BYTES)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,width", [(1, 1, 1), (2, 64, 128), (3, 20, 129), (8, 16, 300)])
def test_plain(fmt, T, H, width):
    c = Case(T, H, width, fmt, seed=fmt + 10 * T)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H,width,length", [(5, 13, 700, 613), (1, 128, 1000, 1000), (32, 64, 513, 400)])
def test_everything_on(fmt, T, H, width, length):
    rope = None if fmt == W.FMT_V32_656 else (W.ROPE_NEOX if T != 5 else W.ROPE_GPTJ)
    c = Case(T, H, width, fmt, seed=T, length=length, invalid=0.1, rope=rope, sink=True, tail=True, page_pad=32)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("sms", [2, 4, 8, 12, 28, 152])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [4, 20])
def test_splits(sms, tail, T):
    """Row tiles whole in a pair, shared by two, cut into many."""
    c = Case(T, 32, 1100, W.FMT_NVFP4_288, seed=sms, sink=True, tail=tail)
    out, lse, attn = c.run(num_sms=sms)
    p = attn.plan
    assert (p.row_tiles, p.key_tiles) == (1 if T == 4 else 5, 5)
    assert p.pairs == min(p.row_tiles * 5, sms // 2)
    c.check(out, lse)


@pytest.mark.parametrize("length", [0, -3, 1, 127, 128, 129, 255, 300, 1 << 20])
@pytest.mark.parametrize("tail", [False, True])
def test_lengths(length, tail):
    c = Case(3, 16, 300, W.FMT_FP8_528, seed=5, length=length, sink=True, tail=tail)
    out, lse, _ = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("tail", [False, True])
def test_no_slot_kept(tail):
    c = Case(3, 16, 300, W.FMT_FP8_528, seed=6, sink=True, tail=tail)
    c.slots.fill_(-1)
    out, lse, _ = c.run()
    c.check(out, lse)
    c = Case(3, 16, 300, W.FMT_FP8_528, seed=7)
    c.slots[:130] = -1                       # the first tile keeps nothing
    c.slots[-30:] = c.cache.num_slots
    out, lse, _ = c.run(num_sms=2)
    c.check(out, lse)


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_FP8_528_UE8M0, W.FMT_MODEL1_584, W.FMT_V32_656])
@pytest.mark.parametrize("mag,q_log2", [((-20,), 20), ((16,), -16), ((0, 3, -2), 0), ((0, 0, 0, 12, -9), -10)])
def test_magnitudes(fmt, mag, q_log2):
    """Rows at 2^k and mixed within a group of 32 keys (one exponent each)."""
    c = Case(4, 32, 400, fmt, seed=11, mag=mag, q_log2=q_log2)
    out, lse, _ = c.run()
    c.check(out, lse)


def test_scores_that_raise_the_maximum():
    """Keys in rising order of their scores: the running maximum moves late."""
    c = Case(2, 64, 1024, W.FMT_FP8_528, seed=12, q_log2=3)
    rec = c.cache.data[:, :64 * 528].reshape(-1, 528).cpu().numpy()
    k = R.record_values(c.fmt, rec[c.slots.cpu().numpy()])
    order = np.argsort((k @ c.q.double().cpu().numpy()[0, 0]))
    c.slots = c.slots[torch.from_numpy(order).cuda()].contiguous()
    for sms in (2, 0):
        out, lse, _ = c.run(num_sms=sms)
        c.check(out, lse)


def test_repeated_slots_and_long_list():
    c = Case(1, 16, 70000, W.FMT_NVFP4_288, seed=13, num_slots=4096)
    out, lse, _ = c.run()
    c.check(out, lse)


def test_many_row_tiles():
    c = Case(97, 128, 260, W.FMT_FP8_528_UE8M0, seed=14, rope=W.ROPE_GPTJ, sink=True, tail=True)
    out, lse, _ = c.run()
    c.check(out, lse)


def test_strided_queries():
    c = Case(4, 16, 200, W.FMT_FP8_528, seed=15)
    wide = torch.zeros((4, 16, 1024), dtype=torch.bfloat16, device="cuda")
    wide[:, :, 512:] = c.q
    c.q = wide[:, :, 512:]
    out, lse, _ = c.run()
    c.check(out, lse)


def test_one_token_of_any_stride():
    c = Case(1, 16, 200, W.FMT_FP8_528, seed=30)
    wide = torch.zeros((16, 1024), dtype=torch.bfloat16, device="cuda")
    wide[:, 512:] = c.q[0]
    c.q = wide[:, 512:].unsqueeze(0)
    out, lse, _ = c.run()
    c.check(out, lse)


def test_nan_query_stays_in_its_row():
    c = Case(3, 16, 300, W.FMT_FP8_528, seed=31)
    c.q[1, 4, 7] = float("nan")
    out, lse, _ = c.run()
    assert bool(torch.isnan(out[1, 4]).all()) and bool(torch.isnan(lse[1, 4]))
    ok = torch.ones((3, 16), dtype=torch.bool, device="cuda")
    ok[1, 4] = False
    assert not bool(torch.isnan(out[ok]).any()) and not bool(torch.isnan(lse[ok]).any())
    c.q[1, 4] = 0
    want, wlse, _ = c.run()
    assert torch.equal(out[ok], want[ok]) and torch.equal(lse[ok], wlse[ok])


@pytest.mark.parametrize("sink", [float("inf"), -float("inf"), 1e30, -1e30])
def test_sinks_at_the_ends(sink):
    c = Case(2, 16, 300, W.FMT_FP8_528, seed=32, sink=True, tail=True)
    c.sink.fill_(sink)
    out, lse, _ = c.run()
    if sink > 0:
        assert bool((out == 0).all())            # all weight on the sink
        c.sink = None
        assert torch.equal(c.run()[1], lse)      # which lse does not contain
    else:
        c.check(out, lse)


def test_negative_and_zero_scale():
    for scale in (-0.05, 0.0):
        c = Case(2, 16, 300, W.FMT_NVFP4_288, seed=33)
        c.scale = scale
        out, lse, _ = c.run()
        r_out, r_lse, tol, ltol = c.reference()
        assert np.all(np.abs(lse.double().cpu().numpy().reshape(-1) - r_lse) <= 0.1 * abs(scale) + 1e-4)
        assert np.abs(out.double().cpu().numpy().reshape(r_out.shape) - r_out).max() <= 2e-2


def test_in_place_tail():
    c = Case(9, 64, 500, W.FMT_FP8_528, seed=16, sink=True, tail=True)
    want_out, want_lse, attn = c.run()
    want_out, want_lse = want_out.clone(), want_lse.clone()
    o, l = c.tail_out.clone(), c.tail_lse.clone()
    B.dsa_prefix_run(attn.plan, attn.workspace, c.q, c.cache, c.slots, c.length, c.sink, None, None, 0, c.scale,
                     o, l, o, l)
    torch.cuda.synchronize()
    assert torch.equal(o.view(torch.int16), want_out.view(torch.int16))
    assert torch.equal(l.view(torch.int32), want_lse.view(torch.int32))


def test_nan_key_reaches_the_output():
    c = Case(2, 16, 300, W.FMT_FP8_528, seed=17)
    c.cache.data[:, :64 * 528].view(-1, 64, 528)[0, 0, 512:528].view(torch.float32).fill_(float("nan"))
    c.slots[200] = 0
    for sms in (2, 0):
        out, lse, _ = c.run(num_sms=sms)
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    c.slots[200] = -1                        # named by no kept entry: not read
    c.slots[c.slots == 0] = -1
    out, lse, _ = c.run()
    c.check(out, lse)


def test_position_outside_the_table_sets_the_status():
    c = Case(2, 16, 200, W.FMT_FP8_528, seed=18, rope=W.ROPE_NEOX)
    c.pos[1] = 4096
    attn = B.PrefixAttention(2, 16, 200, "cuda")
    attn(c.q, c.cache, c.slots, c.length, c.scale, None, c.pos, c.cs)
    assert B.dsa_decode_read_status(attn.workspace) == -1
    c.pos[1] = 0                             # the next call starts from a cleared word
    out, lse, _ = c.run(attn=attn)
    c.check(out, lse)


def test_reproducible_and_captured():
    c = Case(24, 64, 2000, W.FMT_FP8_528, seed=19, rope=W.ROPE_NEOX, sink=True, tail=True)
    out, lse, attn = c.run()
    want = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn(c.q, c.cache, c.slots, c.length, c.scale, c.sink, c.pos, c.cs, c.style, c.tail_out, c.tail_lse)
    for _ in range(3):
        attn.out.fill_(float("nan"))
        attn.lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(attn.out.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(attn.lse.view(torch.int32), want[1].view(torch.int32))
    # a length that changes between replays is read by the kernels
    c.length.fill_(77)
    g.replay()
    torch.cuda.synchronize()
    c.check(attn.out, attn.lse)


def test_two_streams_with_their_own_workspaces():
    cs = [Case(16, 64, 1500, W.FMT_FP8_528, seed=20 + i, sink=True) for i in range(2)]
    want = [tuple(t.clone() for t in c.run()[:2]) for c in cs]
    attn = [B.PrefixAttention(16, 64, 1500, "cuda") for _ in cs]
    st = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, a, s in zip(cs, attn, st):
            a(c.q, c.cache, c.slots, c.length, c.scale, c.sink, stream=s)
    torch.cuda.synchronize()
    for w, a in zip(want, attn):
        assert torch.equal(a.out, w[0]) and torch.equal(a.lse, w[1])


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_FP8_528_UE8M0])
def test_decode_step_behind_a_prefix(fmt):
    """Keys written, own lists decoded, prefix merged: one attention over both."""
    T, H, P = 6, 64, 700
    w = W.make_workload(T=T, H=H, seed=41, sink=True, rope=True, rope_style=W.ROPE_NEOX, device="cuda",
                        swa=dict(width=128, lens=(0, 128), fmt=fmt, page=64, slots=2048))
    c = Case(T, H, P, fmt, seed=42, sink=True)
    rows = torch.randn((P, 512), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    c.slots = torch.randperm(c.cache.num_slots, device="cuda")[:P].to(torch.int32)
    B.dsa_cache_write(c.cache, c.slots, rows)
    sink, w.sink = w.sink, None
    dec = B.Decoder(w)
    tail_out, tail_lse = dec(w)
    attn = B.PrefixAttention(T, H, P, "cuda")
    out, lse = attn(w.q, c.cache, c.slots, c.length, w.scale, sink, w.positions, w.cos_sin, w.rope_style,
                    tail_out, tail_lse)
    torch.cuda.synchronize()
    # one softmax over the two lists, in 64 bits
    kp = R.record_values(fmt, c.cache.data[:, :64 * 528].reshape(-1, 528).cpu().numpy()[c.slots.cpu().numpy()])
    sw = w.swa_cache.data[:, :64 * 528].reshape(-1, 528).cpu().numpy()
    q = R.transform(w.q.double().cpu().numpy().reshape(T * H, 512), positions=np.repeat(w.positions.cpu().numpy(), H),
                    cos_sin=w.cos_sin.cpu().numpy(), style=w.rope_style).reshape(T, H, 512)
    for t in range(T):
        ids = w.swa.ids[t, :int(w.swa.lens[t])].cpu().numpy()
        k = np.concatenate([kp, R.record_values(fmt, sw[ids])])
        s = w.scale * (q[t] @ k.T)
        l = np.log(np.exp(s).sum(1))
        sk = sink.double().cpu().numpy()
        o = (np.exp(s) @ k) / (np.exp(l) + np.exp(sk))[:, None]
        assert np.abs(lse[t].double().cpu().numpy() - l).max() <= 1e-3
        got = out[t].double().cpu().numpy()
        assert np.abs(got - o).max() <= 2e-2
        cos = (got * o).sum(-1) / (np.linalg.norm(got, axis=-1) * np.linalg.norm(o, axis=-1))
        assert cos.min() >= 0.9999


def test_short_wait_budget_reports_a_timeout(monkeypatch):
    """A budget of a few cycles runs out in the kernel's first waits: the call
    ends, the status says so, and the next call with the default budget is
    right."""
    c = Case(8, 64, 1000, W.FMT_FP8_528, seed=50)
    monkeypatch.setenv("DSA_DECODE_WAIT_BUDGET", "1")
    attn = B.PrefixAttention(8, 64, 1000, "cuda")
    monkeypatch.delenv("DSA_DECODE_WAIT_BUDGET")
    attn(c.q, c.cache, c.slots, c.length, c.scale)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == -6
    out, lse, _ = c.run()
    c.check(out, lse)


def test_binding_refuses_what_pointers_cannot_tell():
    c = Case(2, 16, 300, W.FMT_FP8_528, seed=60, rope=W.ROPE_NEOX, sink=True, tail=True)
    want, _, attn = c.run()
    want = want.clone()
    ok = dict(plan=attn.plan, workspace=attn.workspace, q=c.q, cache=c.cache, slots=c.slots, length=c.length, sink=c.sink,
              positions=c.pos, cos_sin=c.cs, rope_style=0, scale=c.scale, tail_out=c.tail_out, tail_lse=c.tail_lse,
              out=attn.out, lse=attn.lse)
    bad = [dict(q=c.q.float()), dict(q=c.q[:1]), dict(q=c.q[:, :8]), dict(q=c.q.transpose(1, 2)), dict(q=c.q.cpu()),
           dict(slots=c.slots[:299]), dict(slots=c.slots.long()), dict(slots=None), dict(length=c.length.long()),
           dict(length=c.length.repeat(2)), dict(length=None), dict(sink=c.sink[:8]), dict(sink=c.sink.double()),
           dict(positions=c.pos.int()), dict(positions=None), dict(cos_sin=c.cs[:, :60]), dict(tail_out=c.tail_out.float()),
           dict(tail_out=None), dict(tail_lse=c.tail_lse[:, :8]), dict(tail_lse=None), dict(out=attn.out.float()),
           dict(out=attn.out[:, :, ::2]), dict(out=None), dict(lse=attn.lse.t()), dict(lse=attn.lse.cpu())]
    for kw in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_prefix_run(**dict(ok, **kw))
        assert e.value.status == -1, kw
    with pytest.raises(B.DsaError) as e:
        B.dsa_prefix_run(**dict(ok, workspace=attn.workspace[:1024]))
    assert e.value.status == -4
    torch.cuda.synchronize()
    assert torch.equal(attn.out, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    B.dsa_prefix_run(**ok, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(attn.out, want)
