"""dsa_weights_run on the GPU against the formulas in 64 bits.

Tolerances. Operands of the products are exact in f16 but for query elements
below 2^-14 of their row's largest, off by 2^-25 of it. The tensor core adds 576
exact products in at most 36 steps, each off by at most 2^-22 of the sum of
magnitudes A: 2^-16 A bounds them. A score in log2 units stays below 2^6, its
fp32 work (two or three roundings, and the exponential's 2^-22) costs below
2^-17 in it. So a weight is off by a factor e^{+-delta}, delta = 2^-16 A + 2^-17
+ the small elements' share; their sum by 2^-20 of itself (a few tens of additions
in a row, partial sums in order); the result is fp32. All of it has either sign:
over a whole list the norm of the errors stays below 2^-17 of the norm."""
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


class Case:
    """A batch with its true lse and scores from before."""

    def __init__(self, *args, base=True, **kw):
        self.c = c = Batch(*args, **kw)
        self.lse = torch.full((c.T, c.H), -INF, dtype=torch.float64, device="cuda")
        for b, t, at, k, x, mass in c.scores():
            if x.shape[2]:
                self.lse[t:t + x.shape[0]] = torch.logsumexp(x, 2)
        self.lse = self.lse.float()
        g = torch.Generator(device="cuda").manual_seed(99)
        self.before = torch.rand((c.B, c.width), generator=g, device="cuda") if base else None

    def call(self, attn, out, **kw):
        c = self.c
        return attn(c.q, c.cache, c.slots, c.lengths, c.starts, self.lse, self.before, out, c.scale, c.window, c.sink, **kw)

    def run(self, num_sms=0, attn=None):
        c = self.c
        attn = attn or B.AttentionWeights(c.T, c.B, c.H, c.width, "cuda", c.d, num_sms)
        out = torch.full((c.B, c.width), 7.0, device="cuda")
        self.call(attn, out)
        torch.cuda.synchronize()
        assert B.dsa_decode_read_status(attn.workspace) == 0
        return out, attn

    def reference(self):
        c = self.c
        want = torch.full((c.B, c.width), 7.0, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        den = self.lse.double()
        if c.sink is not None:
            den = torch.logaddexp(den, c.sink.double())
        den = torch.where(self.lse == -INF, torch.full_like(den, INF), den)
        for b, t, at, k, x, mass in c.scores():
            n, length = x.shape[0], min(max(int(c.lengths[b]), 0), c.width)
            base = torch.zeros(length, dtype=torch.float64, device="cuda") if self.before is None else self.before[b, :length].double()
            want[b, :length] = base
            if n == 0 or len(at) == 0:
                continue
            w = (x - den[t:t + n, :, None]).exp()
            small = c.scale * c.queries()[t:t + n].abs().amax(2)[..., None] * k.abs().sum(1) * 2.0 ** -25
            want[b, at] += w.sum((0, 1))
            tol[b, at] = (w * torch.expm1(2.0 ** -16 * mass + 2.0 ** -17 + abs(small))).sum((0, 1))
        return want, tol + want.abs() * 2.0 ** -20

    def check(self, out):
        want, tol = self.reference()
        got = out.double()
        bad = (got - want).abs() > tol
        assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), float(((got - want).abs() / tol).max()))
        base = torch.zeros_like(want) if self.before is None else self.before.double()
        inner = want != 7.0
        sums = torch.where(inner, want - base, torch.zeros_like(want))
        if float(sums.norm()) > 0:
            rel = float(((got - want)[inner]).norm() / want[inner].norm())
            assert rel <= 2.0 ** -17, rel


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,H", [([(1, 1)], 1), ([(1, 128)], 64), ([(7, 129), (1, 3)], 20), ([(16, 300), (1, 257), (40, 40)], 16)])
def test_plain(fmt, sizes, H):
    c = Case(sizes, H, fmt, seed=fmt, base=False)
    c.check(c.run()[0])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("window", [0, 100, 128])
def test_everything_on(fmt, window):
    c = Case([(33, 700), (1, 513), (0, 90), (5, 5), (90, 612)], 20, fmt, seed=5, width=720, invalid=0.1, sink=True, window=window,
             page_pad=32, before=3, behind=4)
    c.check(c.run()[0])


@pytest.mark.parametrize("H", [1, 8, 16, 31, 32, 33, 64, 65, 96, 128, 129, 200, 256, 300])
@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_NVFP4_288])
def test_single_tokens_of_any_head_count(H, fmt):
    """Steps of 64, 128 and 256 rows, rows that end within them."""
    c = Case([(1, 200), (1, 65), (1, 128)], H, fmt, seed=H, sink=True)
    c.check(c.run()[0])


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 600, 2**31 - 1])
def test_windows(window):
    c = Case([(70, 500), (1, 256), (200, 200)], 16, W.FMT_FP8_528_UE8M0, seed=window % 97, window=window)
    c.check(c.run()[0])


@pytest.mark.parametrize("length", [0, -3, 1, 4, 5, 6, 127, 128, 129, 255, 256, 257, 1 << 20])
@pytest.mark.parametrize("window", [0, 3])
def test_lengths(length, window):
    c = Case([(5, length), (2, 30)], 40, W.FMT_FP8_528, width=300, seed=6, window=window, sink=True)
    c.check(c.run()[0])


@pytest.mark.parametrize("sms", [2, 4, 12, 60, 152])
@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_MODEL1_584])
@pytest.mark.parametrize("window", [0, 60])
def test_rows_shared_by_several_items(sms, fmt, window):
    c = Case([(90, 400), (1, 130), (40, 333)], 64, fmt, seed=sms, sink=True, window=window)
    out, attn = c.run(sms)
    assert {2: attn.plan.splits == 1, 152: attn.plan.splits > 1}.get(sms, 1 <= attn.plan.splits <= 11)
    c.check(out)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,window", [([(100, 260)], 0), ([(100, 2300), (77, 1500)], 0), ([(150, 1200), (120, 120)], 100)])
def test_many_rows_per_key(fmt, sizes, window):
    """128 and 256 keys to an item, whole and in parts."""
    c = Case(sizes, 128, fmt, seed=21, sink=True, window=window, invalid=0.05)
    kinds = set()
    for sms in (2, 8, 0):
        out, attn = c.run(sms)
        c.check(out)
        kinds.add((attn.plan.splits > 1, attn.plan.wide_splits))
    assert len(kinds) > 1


def test_many_sequences_and_items():
    sizes = [(i % 3, 1 + (37 * i) % 200) for i in range(700)]
    c = Case(sizes, 8, W.FMT_NVFP4_288, seed=8, width=200, window=64, sink=True, num_slots=8192)
    c.check(c.run()[0])


@pytest.mark.parametrize("sms", [0, 2])
def test_long_list(sms):
    """Also more items to a pair than it holds in shared memory."""
    c = Case([(1, 70001)], 16, W.FMT_FP8_528, seed=13, num_slots=4096)
    c.check(c.run(sms)[0])


@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_MODEL1_584, W.FMT_V32_656])
@pytest.mark.parametrize("mag,q_log2", [((-20,), 20), ((16,), -16), ((0, 0, 0, 12, -9), -10)])
def test_magnitudes(fmt, mag, q_log2):
    c = Case([(20, 400), (3, 70)], 32, fmt, seed=11, mag=mag, q_log2=q_log2, window=200)
    c.check(c.run()[0])


def test_in_place_strided_and_accumulated():
    c = Case([(4, 200), (6, 150)], 16, W.FMT_FP8_528, seed=15, window=30)
    out, attn = c.run()
    wide = torch.full((2, 333), 5.0, device="cuda")
    wide[:, 7:207] = c.before
    view = wide[:, 7:207]
    q = torch.zeros((c.c.T, 16, 1024), dtype=torch.bfloat16, device="cuda")
    q[:, :, 512:] = c.c.q
    c.c.q, before = q[:, :, 512:], c.before
    c.before = view
    c.call(attn, view)
    torch.cuda.synchronize()
    for b, (_, n) in enumerate(c.c.sizes):
        assert torch.equal(view[b, :n], out[b, :n])
        assert torch.equal(view[b, n:], before[b, n:])
    assert bool((wide[:, :7] == 5).all()) and bool((wide[:, 207:] == 5).all())
    c.call(attn, view)                       # and once more on top
    torch.cuda.synchronize()
    twice = out + (out - before)
    for b, (_, n) in enumerate(c.c.sizes):
        assert float((view[b, :n] - twice[b, :n]).abs().max()) <= 1e-5


def test_negative_scale_and_no_tokens():
    c = Case([(20, 300), (1, 64)], 16, W.FMT_FP8_528, seed=33)
    c.c.scale = -0.03
    for b, t, at, k, x, mass in c.c.scores():
        c.lse[t:t + x.shape[0]] = torch.logsumexp(x, 2).float()
    c.check(c.run()[0])
    c = Case([(0, 30), (0, 0), (0, 200)], 16, W.FMT_FP8_528, seed=4, behind=5)
    out, _ = c.run()
    c.check(out)
    assert torch.equal(out[0, :30], c.before[0, :30]) and torch.equal(out[2, :200], c.before[2, :200])


@pytest.mark.parametrize("H", [1, 20, 64, 65, 100])
@pytest.mark.parametrize("fmt", [W.FMT_FP8_528, W.FMT_NVFP4_288, W.FMT_V32_656])
def test_what_the_workspace_held_does_not_count(H, fmt):
    """Image rows behind a sequence's last one: zeros, or never taken."""
    c = Case([(1, 300), (2, 200), (3, 130), (1, 1), (4, 500)], H, fmt, seed=H, sink=True)
    attn = B.AttentionWeights(c.c.T, c.c.B, H, c.c.width, "cuda", c.c.d)
    for byte in (0xFF, 0x7C):   # NaN, and large numbers and infinities
        attn.workspace.fill_(byte)
        c.check(c.run(attn=attn)[0])


def test_sums_of_all_weights():
    """Every query row's weights add up to one."""
    c = Case([(30, 500), (1, 300)], 64, W.FMT_FP8_528_UE8M0, seed=30, base=False)
    out, _ = c.run()
    for b, (n, length) in enumerate(c.c.sizes):
        assert abs(float(out[b, :length].double().sum()) / (n * 64) - 1) <= 1e-5


@pytest.mark.parametrize("sink", [INF, -INF, 1e30, -1e30])
def test_sinks_at_the_ends(sink):
    c = Case([(2, 300)], 16, W.FMT_FP8_528, seed=32, sink=True)
    c.c.sink.fill_(sink)
    out, _ = c.run()
    if sink > 0:
        assert torch.equal(out, c.before)
    else:
        c.check(out)


def test_rows_without_weights_and_nan():
    c = Case([(3, 200)], 16, W.FMT_FP8_528, seed=33)
    full = c.run()[0]
    c.lse[1, 4] = -INF
    c.check(c.run()[0])
    c.lse[1, 4] = float("nan")
    out, _ = c.run()
    assert bool(torch.isnan(out[0, :199]).all()) and not bool(torch.isnan(out[0, 199]))     # token 1 does not see the last record
    assert not bool(torch.isnan(full).any())


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_key_spoils_its_own_score_only(fmt):
    c = Case([(40, 300)], 16, fmt, seed=17)
    c.c.slots[c.c.slots == 0] = -1
    clean, _ = c.run()
    c.c.slots[0, 270] = 0
    rec = c.c.cache.data[0, :c.c.cache.record_bytes]
    if fmt in (W.FMT_FP8_528, W.FMT_V32_656):
        rec[512:528].view(torch.float32).fill_(float("nan"))
    else:
        rec[:] = 0x7F if fmt == W.FMT_NVFP4_288 else 0xFF
    out, _ = c.run()
    assert bool(torch.isnan(out[0, 270]))
    ok = torch.ones(300, dtype=torch.bool, device="cuda")
    ok[270] = False
    assert torch.equal(out[0, ok], clean[0, ok])


def test_starts_out_of_order_leave_everything():
    c = Case([(3, 300), (4, 200)], 16, W.FMT_FP8_528, seed=18)
    out, attn = c.run()
    starts = c.c.starts
    for bad in ([0, 5, 4], [-1, 3, 7], [0, 3, 8], [2**31 - 1, 3, 7]):
        out.fill_(7.0)
        c.c.starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        c.call(attn, out)
        assert B.dsa_decode_read_status(attn.workspace) == -1
        assert bool((out == 7).all())
    c.c.starts = starts
    c.check(c.run(attn=attn)[0])


def test_reproducible_and_captured():
    c = Case([(60, 900), (1, 1500), (20, 333)], 64, W.FMT_FP8_528, seed=19, sink=True)
    want, attn = c.run()
    out = torch.full_like(want, 7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(attn, out)
    for _ in range(3):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int32), want.view(torch.int32))
    c.c.sizes = [(10, 70), (61, 1400), (10, 10)]
    c.c.lengths.copy_(torch.tensor([70, 1400, 10]))
    c.c.starts.copy_(torch.tensor([0, 10, 71, 81]))
    for b, t, at, k, x, mass in c.c.scores():
        c.lse[t:t + x.shape[0]] = torch.logsumexp(x, 2).float()
    out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    c.check(out)


def test_two_streams_with_their_own_workspaces():
    cs = [Case([(30, 900), (9, 1500)], 64, W.FMT_FP8_528, seed=20 + i, sink=True) for i in range(2)]
    want = [c.run()[0] for c in cs]
    attn = [B.AttentionWeights(c.c.T, c.c.B, c.c.H, c.c.width, "cuda") for c in cs]
    outs = [torch.full_like(w, 7.0) for w in want]
    st = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, a, o, s in zip(cs, attn, outs, st):
            c.call(a, o, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(o, w)


def test_short_wait_budget_reports_a_timeout(monkeypatch):
    c = Case([(40, 1000)], 64, W.FMT_FP8_528, seed=50)
    monkeypatch.setenv("DSA_DECODE_WAIT_BUDGET", "1")
    attn = B.AttentionWeights(c.c.T, c.c.B, c.c.H, c.c.width, "cuda")
    monkeypatch.delenv("DSA_DECODE_WAIT_BUDGET")
    c.call(attn, torch.empty((1, 1000), device="cuda"))
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == -6
    c.check(c.run()[0])


def test_binding_refuses_what_pointers_cannot_tell():
    c = Case([(2, 300), (3, 100)], 16, W.FMT_FP8_528, seed=60, sink=True)
    out, attn = c.run()
    b = c.c
    want = out.clone()
    ok = dict(plan=attn.plan, workspace=attn.workspace, q=b.q, cache=b.cache, slots=b.slots, lengths=b.lengths, starts=b.starts,
              window=0, scale=b.scale, sink=b.sink, lse=c.lse, scores_in=c.before, scores_out=out)
    bad = [dict(q=b.q.float()), dict(q=b.q[:1]), dict(q=b.q.cpu()), dict(q=None), dict(slots=b.slots[:, :299]), dict(slots=b.slots[:1]),
           dict(slots=b.slots.long()), dict(slots=None), dict(lengths=b.lengths[:1]), dict(starts=b.starts[:2]), dict(starts=None),
           dict(window=-1), dict(scale=INF), dict(sink=b.sink[:8]), dict(lse=c.lse[:1]), dict(lse=None), dict(lse=c.lse.double()),
           dict(scores_in=c.before[:, :10]), dict(scores_in=c.before.double()), dict(scores_out=None), dict(scores_out=out[:1]),
           dict(scores_out=out.t())]
    for kw in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_weights_run(**dict(ok, **kw))
        assert e.value.status == -1, kw
    with pytest.raises(B.DsaError) as e:
        B.dsa_weights_run(**dict(ok, workspace=attn.workspace[:1024]))
    assert e.value.status == -4
    torch.cuda.synchronize()
    assert torch.equal(out, want)
