"""dsa_evict on the GPU against a plain sort: every slot, score and count equal."""
import math
import random

import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


def choose(scores, budget, first, last):
    """List positions that stay."""
    n = len(scores)
    if n <= budget:
        return list(range(n))
    lo = min(first, budget)
    hi = n - min(last, budget - lo)
    rank = lambda i: (1, 0.0, i) if math.isnan(scores[i]) else (0, -scores[i], i)
    middle = sorted(range(lo, hi), key=rank)[:budget - lo - (n - hi)]
    return sorted(list(range(lo)) + middle + list(range(hi, n)))


class Lists:
    def __init__(self, lengths, width, budget, first=0, last=0, seed=0, scores=None, pad=0):
        g = torch.Generator().manual_seed(seed)
        n, self.budget, self.first, self.last, self.width = len(lengths), budget, first, last, width
        most = min(budget, width)
        self.slots = torch.randperm(n * width, generator=g).view(n, width).to(torch.int32).cuda()
        self.scores = (torch.exp(3 * torch.randn((n, width), generator=g)) if scores is None else scores).float().cuda()
        self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.kept = torch.full((n, most + pad), -7, dtype=torch.int32, device="cuda")
        self.kept_scores = torch.full((n, most + pad), -7.0, device="cuda")
        self.kept_lengths = torch.full((n,), -7, dtype=torch.int32, device="cuda")
        self.freed = torch.full((n, width - most + pad), -7, dtype=torch.int32, device="cuda")
        self.freed_counts = torch.full((n,), -7, dtype=torch.int32, device="cuda")

    def call(self, **kw):
        B.dsa_evict(self.slots, self.lengths, self.scores, self.budget, self.kept, self.kept_scores, self.kept_lengths, self.freed,
                    self.freed_counts, self.first, self.last, **kw)

    def check(self):
        torch.cuda.synchronize()
        bits = self.scores.cpu().view(torch.int32)
        for b, n in enumerate(self.lengths.tolist()):
            n = min(max(n, 0), self.width)
            keep = choose(self.scores[b, :n].tolist(), self.budget, self.first, self.last)
            gone = torch.tensor(sorted(set(range(n)) - set(keep)), dtype=torch.long)
            keep = torch.tensor(keep, dtype=torch.long)
            slots = self.slots[b].cpu()
            assert int(self.kept_lengths[b]) == len(keep) and int(self.freed_counts[b]) == len(gone)
            for got, want in ((self.kept[b].cpu(), slots[keep]), (self.freed[b].cpu(), slots[gone])):
                assert torch.equal(got[:len(want)], want) and bool((got[len(want):] == -7).all())
            got = self.kept_scores[b].cpu()
            assert torch.equal(got[:len(keep)].view(torch.int32), bits[b][keep]) and bool((got[len(keep):] == -7).all())


@pytest.mark.parametrize("width", [1, 2, 31, 32, 33, 500, 2048, 2049, 4097, 9000, 20011])
@pytest.mark.parametrize("share", [0.0, 0.3, 0.9, 1.0])
def test_widths(width, share):
    rng = random.Random(width)
    budget = max(1, int(width * share))
    lengths = [0, width, rng.randint(0, width), budget, min(width, budget + 1), -4, 1 << 30]
    c = Lists(lengths, width, budget, seed=width)
    c.call()
    c.check()


@pytest.mark.parametrize("first,last", [(4, 0), (0, 128), (4, 128), (300, 10), (10, 300), (250, 250), (300, 300), (299, 0),
                                        (1 << 30, 1 << 30)])
def test_protected_ends(first, last):
    c = Lists([2000, 301, 300, 2047], 2047, 300, first, last, seed=(first + last) % 1000)
    c.call()
    c.check()


@pytest.mark.parametrize("kind", ["equal", "zeros", "few", "signs", "nan", "inf", "subnormal", "close", "rising", "falling"])
@pytest.mark.parametrize("width", [777, 9000])
def test_scores(kind, width):
    """Ties go to the lowest position, across warps and CTAs; -0 ties with 0."""
    g = torch.Generator().manual_seed(5)
    r = torch.randint(0, 1 << 20, (3, width), generator=g)
    x = {"equal": torch.full((3, width), 2.5), "zeros": torch.where(r % 2 == 0, -0.0, 0.0), "few": (r % 3).float(),
         "signs": torch.randn((3, width), generator=g), "nan": torch.where(r % 3 == 0, torch.tensor(NAN), (r % 5).float()),
         "inf": torch.where(r % 3 == 0, torch.tensor(INF), torch.where(r % 3 == 1, torch.tensor(-INF), torch.tensor(NAN))),
         "subnormal": r.float() * 2.0 ** -149, "close": 1 + (r % 4096).float() * 2.0 ** -23,
         "rising": torch.arange(width).float().repeat(3, 1), "falling": -torch.arange(width).float().repeat(3, 1)}[kind]
    for first, last in ((0, 0), (7, 40)):
        c = Lists([width, width - 5, width // 2], width, width // 3, first, last, scores=x, pad=3)
        c.call()
        c.check()


def test_lists_past_what_the_shared_memory_holds():
    width = 8 * 40960 + 123
    g = torch.Generator().manual_seed(1)
    c = Lists([width, width - 1], width, 5000, 4, 64, scores=torch.randint(0, 1 << 16, (2, width), generator=g).float())
    c.call()
    c.check()


def test_strided_lists_and_no_freed():
    c = Lists([900, 1000], 1000, 300, 4, 8, seed=9)
    wide = torch.zeros((2, 1111), dtype=torch.int32, device="cuda")
    wide[:, 11:1011] = c.slots
    ws = torch.zeros((2, 1113), device="cuda")
    ws[:, 13:1013] = c.scores
    c.slots, c.scores = wide[:, 11:1011], ws[:, 13:1013]
    c.call()
    c.check()
    want = c.kept.clone()
    c.kept.fill_(-7)
    B.dsa_evict(c.slots, c.lengths, c.scores, 300, c.kept, c.kept_scores, c.kept_lengths, keep_first=4, keep_last=8)
    torch.cuda.synchronize()
    assert torch.equal(c.kept, want)


def test_many_lists_captured():
    rng = random.Random(2)
    c = Lists([rng.randint(0, 5000) for _ in range(300)], 5000, 1200, 4, 100, seed=11)
    c.call()
    torch.cuda.synchronize()
    want = [t.clone() for t in (c.kept, c.kept_scores, c.kept_lengths, c.freed, c.freed_counts)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call()
    for t in (c.kept, c.kept_scores, c.kept_lengths, c.freed, c.freed_counts):
        t.fill_(-7)
    g.replay()
    c.check()
    for t, w in zip((c.kept, c.kept_scores, c.kept_lengths, c.freed, c.freed_counts), want):
        assert torch.equal(t, w)


def test_binding_refuses_what_pointers_cannot_tell():
    c = Lists([100, 90], 100, 30, seed=1)
    ok = dict(slots=c.slots, lengths=c.lengths, scores=c.scores, budget=30, kept_slots=c.kept, kept_scores=c.kept_scores,
              kept_lengths=c.kept_lengths, freed=c.freed, freed_counts=c.freed_counts)
    bad = [dict(slots=c.slots.long()), dict(slots=c.slots[0]), dict(slots=c.slots.t()), dict(slots=c.slots.cpu()), dict(slots=c.slots[:, :99]),
           dict(lengths=c.lengths[:1]), dict(scores=c.scores.double()), dict(scores=c.scores[:1]), dict(budget=0), dict(budget=31),
           dict(budget=29), dict(budget=2**31), dict(keep_first=-1), dict(keep_last=-1), dict(kept_slots=c.kept[:, :29]),
           dict(kept_scores=c.kept_scores[:, :29]), dict(kept_lengths=c.kept_lengths[:1]), dict(freed=None), dict(freed_counts=None),
           dict(freed=c.freed[:, :69]), dict(kept_slots=c.slots), dict(kept_scores=c.scores), dict(freed=c.slots)]
    for kw in bad:
        with pytest.raises(B.DsaError) as e:
            B.dsa_evict(**dict(ok, **kw))
        assert e.value.status == -1, kw
    torch.cuda.synchronize()
    assert bool((c.kept == -7).all()) and bool((c.freed == -7).all())
