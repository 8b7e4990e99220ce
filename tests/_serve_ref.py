"""Plain 64-bit forms of the prompt operators, sequence by sequence (torch on
the tensors' device, written from the definitions in the header). Test
infrastructure; shares nothing with the library."""
import torch

from swa_paged_decode_gb300 import workloads as W
from tests import _cache_ref as R


class Batch:
    """Sequences of new tokens over one cache: sizes = [(new tokens, list
    length)]; lists of ``width`` entries."""

    def __init__(self, sizes, H, fmt, *, width=None, seed=0, page=64, invalid=0.0, rope=None, sink=False, tail=False,
                 window=0, mag=(0,), q_log2=0, page_pad=0, before=0, behind=0, num_slots=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.H, self.fmt, self.window = list(sizes), H, fmt, window
        self.B, self.d = len(sizes), 576 if fmt == W.FMT_V32_656 else 512
        self.width = width or max([1] + [n for _, n in sizes])
        num_slots = num_slots or -(-(self.B * self.width + 64) // page) * page
        self.cache = W.make_cache(num_slots, page, fmt, g, "cuda", page_pad, mag=mag)
        if self.B * self.width <= num_slots:
            ids = torch.randperm(num_slots, generator=g, device="cuda")[:self.B * self.width]
        else:
            ids = torch.randint(0, num_slots, (self.B * self.width,), generator=g, device="cuda")
        self.slots = ids.to(torch.int32).view(self.B, self.width)
        if invalid:
            drop = torch.rand(self.slots.shape, generator=g, device="cuda")
            self.slots[drop < invalid] = -1
            self.slots[drop > 1 - invalid / 2] = num_slots
        self.lengths = torch.tensor([n for _, n in sizes], dtype=torch.int32, device="cuda")
        st = [before]
        for n, _ in sizes:
            st.append(st[-1] + n)
        self.T = st[-1] + behind
        self.starts = torch.tensor(st, dtype=torch.int32, device="cuda")
        self.q = (torch.randn((self.T, H, self.d), generator=g, device="cuda") * 2.0 ** q_log2).to(torch.bfloat16)
        self.scale = self.d ** -0.5
        self.sink = torch.randn((H,), generator=g, device="cuda") if sink else None
        self.tail_out = self.tail_lse = None
        if tail:
            self.tail_out = (0.3 * torch.randn((self.T, H, 512), generator=g, device="cuda")).to(torch.bfloat16)
            self.tail_lse = 3 + 2 * torch.randn((self.T, H), generator=g, device="cuda")
            if self.T * H > 2:
                self.tail_lse.view(-1)[1] = -float("inf")     # a row without a tail
                self.tail_out.view(-1, 512)[1] = float("nan")
        self.style = rope or 0
        self.pos = self.cs = None
        if rope is not None:
            self.cs = W.rope_table(4096, "cuda")
            self.pos = torch.randint(0, 4096, (self.T,), generator=g, device="cuda")

    def records(self):
        rb = self.cache.record_bytes
        return self.cache.data[:, :self.cache.page_size * rb].reshape(-1, rb)

    def queries(self):
        """[T, H, d] in 64 bits, rotated."""
        q = self.q.double()
        if self.pos is None:
            return q
        x = R.transform(q.cpu().numpy().reshape(-1, self.d), positions=self.pos.repeat_interleave(self.H).cpu().numpy(),
                        cos_sin=self.cs.cpu().numpy(), style=self.style)
        return torch.from_numpy(x).cuda().view(self.T, self.H, self.d)

    def scores(self):
        """Of every sequence: (b, its first token, list positions of its kept
        records, their values, scores [n, H, kept] (-inf: not attended), the
        sums of the products' magnitudes)."""
        rec, q = self.records(), self.queries()
        t = int(self.starts[0])
        for b, (n, _) in enumerate(self.sizes):
            length = min(max(int(self.lengths[b]), 0), self.width)
            ids = self.slots[b, :length].long()
            at = ((ids >= 0) & (ids < len(rec))).nonzero()[:, 0]
            k = torch.from_numpy(R.record_values(self.fmt, rec[ids[at]].cpu().numpy())).cuda() if len(at) else q.new_zeros((0, self.d))
            x = self.scale * (q[t:t + n] @ k.T)
            mass = abs(self.scale) * (q[t:t + n].abs() @ k.abs().T)
            p = torch.arange(n, device="cuda")[:, None] + (length - n)
            blind = at[None, :] > p
            if self.window:
                blind = blind | (at[None, :] + self.window <= p)
            yield b, t, at, k, x.masked_fill(blind[:, None, :], -float("inf")), mass.masked_fill(blind[:, None, :], 0.0)
            t += n
