"""The prompt calls as a server makes them, in sequence on one cache: queries
and keys prepared (dsa_qk_norm), attended to (dsa_chunk_run), the records' weights
summed (dsa_weights_run), lists cut (dsa_evict), freed slots used again by the
next tokens, single tokens behind chunks. Every stage is compared with the plain
64-bit forms on what the stage before left."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests import test_chunk_gpu as CH
from tests import test_qk_gpu as QK
from tests import test_weights_gpu as WT
from tests._serve_ref import Batch
from tests.test_evict_gpu import choose

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


class Server:
    def __init__(self, fmt, H, seqs, width, window, page=64):
        self.fmt, self.H, self.window, self.width = fmt, H, window, width
        self.d = 576 if fmt == W.FMT_V32_656 else 512
        pages = 2 * seqs * width // page
        self.cache = W.PagedCache(torch.zeros((pages, page * W.RECORD_BYTES[fmt]), dtype=torch.uint8, device="cuda"), page, fmt)
        self.g = torch.Generator(device="cuda").manual_seed(fmt + 1)
        self.free = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2)).tolist()
        self.lists = [[] for _ in range(seqs)]
        self.at = [0] * seqs                      # the next token's position
        self.scores = torch.zeros((seqs, width), device="cuda")
        self.table = W.rope_table(4096, "cuda")
        self.weight = [1 + 0.1 * torch.randn((512,), generator=self.g, device="cuda") for _ in range(2)]
        self.sink = torch.randn((H,), generator=self.g, device="cuda")

    def step(self, counts):
        """New tokens for every sequence."""
        T, S = sum(counts), len(counts)
        slots, pos = [], []
        for b, n in enumerate(counts):
            new = [self.free.pop() for _ in range(n)]
            self.lists[b] += new
            slots += new
            pos += range(self.at[b], self.at[b] + n)
            self.at[b] += n
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        c = Batch.__new__(Batch)
        c.sizes = [(n, len(l)) for n, l in zip(counts, self.lists)]
        c.H, c.fmt, c.window, c.B, c.d, c.T, c.width = self.H, self.fmt, self.window, S, self.d, T, self.width
        c.cache, c.scale, c.sink = self.cache, self.d ** -0.5, self.sink
        c.pos = c.cs = c.tail_out = c.tail_lse = None
        c.style = 0
        c.slots = i32([l + [-1] * (self.width - len(l)) for l in self.lists])
        c.lengths = i32([len(l) for l in self.lists])
        c.starts = i32([sum(counts[:b]) for b in range(S + 1)])
        raw = torch.randn((T, self.H, self.d), generator=self.g, device="cuda").to(torch.bfloat16)
        keys = torch.randn((T, self.d), generator=self.g, device="cuda").to(torch.bfloat16)
        positions = torch.tensor(pos, device="cuda")
        c.q = torch.empty_like(raw)
        B.dsa_qk_norm(raw, c.q, self.weight[0], keys, self.weight[1], self.cache, i32(slots), 1e-6, positions, self.table)
        out, lse = B.ChunkAttention(T, S, self.H, self.width, "cuda", self.d)(
            c.q, self.cache, c.slots, c.lengths, c.starts, c.scale, self.window, self.sink)
        before = self.scores.clone()
        B.AttentionWeights(T, S, self.H, self.width, "cuda", self.d)(
            c.q, self.cache, c.slots, c.lengths, c.starts, lse, self.scores, self.scores, c.scale, self.window, self.sink)
        torch.cuda.synchronize()
        QK.check(c.q, *QK.reference(raw, self.weight[0], 1e-6, positions, self.table, 0))
        CH.check(c, out, lse)
        w = WT.Case.__new__(WT.Case)
        w.c, w.lse, w.before = c, lse, before
        got = self.scores.clone()
        for b, l in enumerate(self.lists):         # entries behind the lists: as they were
            assert torch.equal(got[b, len(l):], before[b, len(l):])
            got[b, len(l):] = 7
        w.check(got)

    def evict(self, budget, first, last):
        S = len(self.lists)
        slots = torch.tensor([l + [-1] * (self.width - len(l)) for l in self.lists], dtype=torch.int32, device="cuda")
        lengths = torch.tensor([len(l) for l in self.lists], dtype=torch.int32, device="cuda")
        kept = torch.full_like(slots, -1)
        scores = torch.zeros_like(self.scores)
        klen, fcount = torch.zeros_like(lengths), torch.zeros_like(lengths)
        freed = torch.full_like(slots, -1)
        B.dsa_evict(slots, lengths, self.scores, budget, kept, scores, klen, freed, fcount, first, last)
        torch.cuda.synchronize()
        for b, l in enumerate(self.lists):
            keep = choose(self.scores[b, :len(l)].tolist(), budget, first, last)
            gone = [l[i] for i in sorted(set(range(len(l))) - set(keep))]
            self.lists[b] = [l[i] for i in keep]
            assert kept[b, :len(keep)].tolist() == self.lists[b] and int(klen[b]) == len(keep)
            assert freed[b, :len(gone)].tolist() == gone and int(fcount[b]) == len(gone)
            assert torch.equal(scores[b, :len(keep)], self.scores[b, keep])
            self.free += gone
        self.scores = scores


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
@pytest.mark.parametrize("window", [0, 100])
def test_prompt_chunks_eviction_and_single_tokens(fmt, window):
    s = Server(fmt, 32, 3, 600, window)
    s.step([130, 7, 64])
    s.step([200, 1, 0])
    s.evict(150, 4, 32)
    s.step([33, 90, 128])
    s.evict(120, 4, 64)
    for _ in range(2):
        s.step([1, 1, 1])
    assert [len(l) for l in s.lists] == [122, 100, 122]


def test_a_captured_step_follows_its_lists():
    """One graph of attention and weights, replayed as lists, lengths and starts
    change in place."""
    s = Server(W.FMT_FP8_528_UE8M0, 64, 2, 400, 0)
    s.step([100, 60])
    T, S = 20, 2
    q = torch.randn((T, 64, 512), generator=s.g, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([l + [-1] * (400 - len(l)) for l in s.lists], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 10, 20], dtype=torch.int32, device="cuda")
    attn = B.ChunkAttention(T, S, 64, 400, "cuda")
    weights = B.AttentionWeights(T, S, 64, 400, "cuda")
    sums = torch.zeros((S, 400), device="cuda")

    def call():
        attn(q, s.cache, slots, lengths, starts, 0.04, 0, s.sink)
        weights(q, s.cache, slots, lengths, starts, attn.lse, None, sums, 0.04, 0, s.sink)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for sizes, st in (([(10, 100), (10, 60)], [0, 10, 20]), ([(1, 90), (15, 33)], [2, 3, 18]), ([(0, 5), (20, 20)], [0, 0, 20])):
        lengths.copy_(torch.tensor([n for _, n in sizes]))
        starts.copy_(torch.tensor(st))
        attn.out.fill_(7.0)
        attn.lse.fill_(7.0)
        sums.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        c = Batch.__new__(Batch)
        c.sizes, c.H, c.fmt, c.window, c.B, c.d, c.T, c.width = sizes, 64, s.fmt, 0, S, 512, T, 400
        c.cache, c.scale, c.sink, c.pos, c.cs, c.tail_out, c.tail_lse, c.style = s.cache, 0.04, s.sink, None, None, None, None, 0
        c.q, c.slots, c.lengths, c.starts = q, slots, lengths, starts
        CH.check(c, attn.out, attn.lse)
        w = WT.Case.__new__(WT.Case)
        w.c, w.lse, w.before = c, attn.lse, None
        w.check(sums)


def test_records_beyond_four_gigabytes():
    n = 9_000_000
    cache = W.PagedCache(torch.zeros((n // 64, 64 * 528), dtype=torch.uint8, device="cuda"), 64, W.FMT_FP8_528)
    assert cache.data.numel() > 2 ** 32
    c = Batch([(40, 300), (1, 200)], 16, W.FMT_FP8_528, seed=3, sink=True)
    top = torch.arange(cache.num_slots - 600, cache.num_slots, device="cuda", dtype=torch.int32)
    c.slots = top[torch.randperm(600, device="cuda")].view(2, 300)
    keys = torch.randn((600, 512), device="cuda").to(torch.bfloat16)
    q = c.q.clone()
    B.dsa_qk_norm(torch.randn((600, 16, 512), device="cuda").to(torch.bfloat16), torch.empty((600, 16, 512), dtype=torch.bfloat16, device="cuda"),
                  keys=keys, cache=cache, slots=top)
    # the same records in a small cache, under the slots counted from the first of them
    small = W.PagedCache(torch.zeros((10, 64 * 528), dtype=torch.uint8, device="cuda"), 64, W.FMT_FP8_528)
    B.dsa_cache_write(small, top - top[0], keys)
    big = c.slots
    c.cache, c.slots = small, (big - top[0]).contiguous()
    out, lse, _ = CH.run(c)
    want = out.clone(), lse.clone()
    CH.check(c, *want)
    attn = CH.attention(c)
    o2, l2 = attn(q, cache, big, c.lengths, c.starts, c.scale, 0, c.sink)
    s1 = torch.zeros((2, 300), device="cuda")
    s2 = torch.zeros((2, 300), device="cuda")
    call = B.AttentionWeights(c.T, 2, 16, 300, "cuda")
    call(q, cache, big, c.lengths, c.starts, lse, None, s2, c.scale, sink=c.sink)
    call(q, small, c.slots, c.lengths, c.starts, lse, None, s1, c.scale, sink=c.sink)
    torch.cuda.synchronize()
    assert torch.equal(o2, want[0]) and torch.equal(l2, want[1]) and torch.equal(s1, s2) and float(s1.abs().max()) > 0
