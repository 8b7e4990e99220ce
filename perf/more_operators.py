"""The measured cases of the prompt and cache-budget operators.

Four operators that serve a prompt next to the paged decode, in the order in
which a step calls them:

  * query and key norm: queries RMS-normed per head and rotated, each token's
    key likewise and quantized into its record of the cache, in one pass;
  * chunk attention: the new tokens of several sequences (a prompt's chunk, or
    one token) over each sequence's own paged list, causal, with an optional
    sliding window, sink and tail state;
  * attention weights: the weight that each cached record received from the new
    tokens, added to what it had received before;
  * eviction: every list cut to a budget of records by those sums.

``run`` computes a case in its plain form (elementary torch operations, 32
bits or more) or, with ``own`` set, by the package's calls.
"""
import math
import random

import torch

own = False

DIM = 512
ROPE_ROWS = 131072
EPS = 1e-6
NEOX, GPTJ = 0, 1
FORMATS = {"fp8_528": 0, "nvfp4_288": 1, "fp8_528_ue8m0": 2, "model1_584": 3, "v32_656": 4}
RECORD = {"fp8_528": 528, "nvfp4_288": 288, "fp8_528_ue8m0": 528, "model1_584": 584, "v32_656": 656}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dims(fmt):
    """Dims of a key: V3.2 records carry 64 more than the value."""
    return 576 if fmt == "v32_656" else DIM


def listed():
    return [
        # a decode step of 32 requests prepares its queries and keys (latency counts)
        dict(name="norm_step_fp8", op="norm", fmt="fp8_528", T=32, H=64, type="bf16", page=64, rope=NEOX, norm=True, pad=0.1),
        # a large chunk of prompts: 2 GB of queries in and out
        dict(name="norm_prefill_model1", op="norm", fmt="model1_584", T=8192, H=128, type="bf16", page=64, rope=GPTJ, norm=True, pad=0.0),
        # the first tokens of two short prompts (latency counts)
        dict(name="chunk_small_fp8", op="chunk", fmt="fp8_528", seqs=2, singles=0, tokens=16, context=512, ragged=0, H=16, page=64,
             window=0, rope=NEOX, sink=False, tail=False, invalid=0.0),
        # four prompts through a sliding-window layer, odd lengths
        dict(name="chunk_window_ue8m0", op="chunk", fmt="fp8_528_ue8m0", seqs=4, singles=0, tokens=1100, context=2100, ragged=5, H=64, page=64,
             window=128, rope=GPTJ, sink=True, tail=False, invalid=0.0),
        # continuous batching: decoding requests and two prompts' chunks in one call
        dict(name="chunk_mixed_nvfp4", op="chunk", fmt="nvfp4_288", seqs=26, singles=24, tokens=512, context=8192, ragged=7, H=64, page=256,
             window=0, rope=NEOX, sink=True, tail=False, invalid=0.0),
        # odd counts of everything, unused slots, merged with the state of another list
        dict(name="chunk_ragged_v32", op="chunk", fmt="v32_656", seqs=5, singles=1, tokens=91, context=1501, ragged=11, H=20, page=64,
             window=0, rope=-1, sink=True, tail=True, invalid=0.03),
        # a chunk at the end of a long prompt in the widest layer
        dict(name="chunk_long_fp8", op="chunk", fmt="fp8_528", seqs=1, singles=0, tokens=1024, context=16384, ragged=0, H=128, page=64,
             window=0, rope=NEOX, sink=True, tail=False, invalid=0.0),
        # a decode step adds its weights to the records' sums
        dict(name="weights_step_fp8", op="weights", fmt="fp8_528", seqs=32, singles=32, tokens=1, context=4096, ragged=3, H=64, page=64,
             window=0, sink=True, invalid=0.0),
        # the last 32 tokens of four prompts vote on their records
        dict(name="weights_observe_ue8m0", op="weights", fmt="fp8_528_ue8m0", seqs=4, singles=0, tokens=32, context=8192, ragged=9, H=64, page=64,
             window=0, sink=False, invalid=0.02),
        # a long document, 64 observing tokens of the widest layer
        dict(name="weights_long_model1", op="weights", fmt="model1_584", seqs=1, singles=0, tokens=64, context=65536, ragged=0, H=128, page=64,
             window=0, sink=True, invalid=0.0),
        # a batch of requests goes over its budget (latency counts)
        dict(name="evict_step", op="evict", seqs=32, context=2048, ragged=13, budget=1024, first=4, last=128),
        # long prompts cut to an eighth, odd lengths
        dict(name="evict_prompt", op="evict", seqs=16, context=65521, ragged=17, budget=8190, first=4, last=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "chunk", "chunk", "chunk", "weights", "weights", "evict"])
    page, ragged = rng.choice([16, 64, 128, 256]), rng.randrange(1, 1 << 20)
    if op == "norm":
        # (records with 4-bit codes are left to the cache write's own cases)
        fmt = rng.choice([f for f in FORMATS if f != "nvfp4_288"])
        while True:
            T, H = _log(rng, 1, 16384), rng.choice([1, 8, 16, 20, 32, 40, 64, 128])
            if T * H <= 8192 * 128:
                break
        return dict(op=op, fmt=fmt, T=T, H=H, type=rng.choice(list(TYPES)), page=page, rope=rng.choice([-1, NEOX, GPTJ]),
                    norm=rng.random() < 0.8, pad=rng.choice([0.0, 0.1]))
    if op == "evict":
        while True:
            seqs, context = _log(rng, 1, 64), _log(rng, 16, 65536)
            if seqs * context <= 16 * 65521:
                break
        budget = max(1, int(context * rng.uniform(0.05, 0.9)))
        return dict(op=op, seqs=seqs, context=context, ragged=ragged, budget=budget, first=rng.choice([0, 4, 16]), last=rng.choice([0, 32, 128]))
    fmt = rng.choice(list(FORMATS))
    H = rng.choice([8, 16, 20, 32, 40, 64, 96, 128])
    while True:
        seqs = _log(rng, 1, 32)
        singles = rng.choice([0, 0, seqs // 2, seqs])
        tokens = _log(rng, 1, 2048 if op == "chunk" else 64)
        context = max(tokens, _log(rng, 64, 65536))
        rows = H * (singles + (seqs - singles) * tokens)
        most = 128 * 1024 * 16384 if op == "chunk" else 128 * 64 * 65536
        if rows * context <= most and seqs * context <= 1 << 18 and rows <= 1 << 19:
            break
    case = dict(op=op, fmt=fmt, seqs=seqs, singles=singles, tokens=tokens, context=context, ragged=ragged, H=H, page=page,
                window=rng.choice([0, 0, 128, _log(rng, 16, 4096)]), sink=rng.random() < 0.5, invalid=rng.choice([0.0, 0.0, 0.03]))
    if op == "chunk":
        case.update(rope=-1 if fmt == "v32_656" else rng.choice([-1, NEOX, GPTJ]), tail=rng.random() < 0.4)
    return case


def shape(case):
    """(new tokens, list length) of every sequence; the length counts them."""
    rng, out = random.Random(case["ragged"]), []
    for i in range(case["seqs"]):
        n, length = (1 if i < case["singles"] else case["tokens"]), case["context"]
        if case["ragged"]:
            n = rng.randint((n + 1) // 2, n)
            length = rng.randint(max(n, length // 2), length)
        out.append((n, length))
    return out


# ------------------------------------------------------------------ inputs

def _table(device):
    """[rows, 64] rows of 32 cosines and 32 sines, angles in 64 bits."""
    w = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=device) / 32.0)
    a = torch.arange(ROPE_ROWS, dtype=torch.float64, device=device)[:, None] * w
    return torch.cat([a.cos(), a.sin()], 1).float()


def _normal(g, *size):
    return torch.randn(size, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (_prepare_evict if case["op"] == "evict" else _prepare_norm if case["op"] == "norm" else _prepare_attend)(case, g)


def _prepare_evict(case, g):
    n, width = case["seqs"], case["context"]
    rng = random.Random(case["ragged"])
    lengths = [rng.randint(width // 2, width) for _ in range(n)]
    s = dict(case=case, lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    s["slots"] = torch.randperm(n * width, generator=g, device="cuda").reshape(n, width).to(torch.int32)
    # sums of softmax weights: heavy-tailed, small ones as good as equal, some records never attended
    w = torch.exp(3.0 * _normal(g, n, width))
    w = torch.where(w < 0.05, torch.round(w * 256.0) / 256.0, w)
    s["scores"] = torch.where(torch.rand((n, width), generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
    k = min(case["budget"], width)
    s["kept"] = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
    s["kept_scores"] = torch.zeros((n, k), device="cuda")
    s["kept_lengths"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    s["freed"] = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    s["freed_counts"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    return s


def _prepare_norm(case, g):
    T, H, fmt, page = case["T"], case["H"], case["fmt"], case["page"]
    d, slots = dims(fmt), -(-T // page) * page
    s = dict(case=case, q=_normal(g, T, H, d).to(TYPES[case["type"]]), keys=(2.0 * _normal(g, T, d)).to(TYPES[case["type"]]))
    s["out"] = torch.empty((T, H, d), dtype=torch.bfloat16, device="cuda")
    s["q_weight"] = 1.0 + 0.1 * _normal(g, DIM) if case["norm"] else None
    s["k_weight"] = 1.0 + 0.1 * _normal(g, DIM) if case["norm"] else None
    s["data"] = torch.zeros((slots // page, page * RECORD[fmt]), dtype=torch.uint8, device="cuda")
    ids = _paged(T, slots, page, g)
    s["slots"] = torch.where(torch.rand(T, generator=g, device="cuda") < case["pad"], torch.full_like(ids, -1), ids)
    s["positions"] = s["table"] = None
    if case["rope"] >= 0:
        s["positions"] = torch.randint(0, ROPE_ROWS, (T,), generator=g, device="cuda")
        s["table"] = _table("cuda")
    if own:
        from swa_paged_decode_gb300 import workloads as W
        s["cache"] = W.PagedCache(s["data"], page, FORMATS[fmt])
    return s


def _paged(n, num_slots, page, g):
    """n distinct slots as an allocator hands them out: whole pages in any
    order, their slots in sequence."""
    pages = torch.randperm(num_slots // page, generator=g, device="cuda")[: -(-n // page)]
    return (pages[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n].to(torch.int32)


def _prepare_attend(case, g):
    fmt, page, H, B, width = case["fmt"], case["page"], case["H"], case["seqs"], case["context"]
    sizes = shape(case)
    T, d = sum(n for n, _ in sizes), dims(fmt)
    per = -(-width // page) * page            # slots of a sequence
    num = B * per
    rec = torch.empty((num, RECORD[fmt]), dtype=torch.uint8, device="cuda")
    for a in range(0, num, 1 << 16):
        b = min(num, a + (1 << 16))
        rec[a:b] = _encode(fmt, _normal(g, b - a, d).double())
    s = dict(case=case, sizes=sizes, data=rec.view(num // page, page * RECORD[fmt]), num_slots=num, scale=d ** -0.5)
    ids = _paged(num, num, page, g).view(B, per)[:, :width].contiguous()
    if case["invalid"]:
        ids = torch.where(torch.rand(ids.shape, generator=g, device="cuda") < case["invalid"], torch.full_like(ids, -1), ids)
    s["slots"] = ids
    s["lengths"] = torch.tensor([n for _, n in sizes], dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([sum(n for n, _ in sizes[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    s["q"] = _normal(g, T, H, d).to(torch.bfloat16)
    s["sink"] = _normal(g, H) if case["sink"] else None
    s["positions"] = s["table"] = s["tail_out"] = s["tail_lse"] = None
    if case["op"] == "chunk":
        if case["rope"] >= 0:
            s["positions"] = torch.cat([torch.arange(n, device="cuda") + (length - n) for n, length in sizes])
            s["table"] = _table("cuda")
        if case["tail"]:   # the state that attention over another list left
            s["tail_out"] = (0.2 * _normal(g, T, H, DIM)).to(torch.bfloat16)
            s["tail_lse"] = 5.0 + _normal(g, T, H)
    else:
        s["lse"] = torch.empty((T, H), device="cuda")   # as the attention of these tokens left it
        for rows, _, x in _scores(s):
            s["lse"].view(-1)[rows] = torch.logsumexp(x, 1)
        s["before"] = torch.exp(_normal(g, B, width))
        s["sums"] = torch.zeros((B, width), device="cuda")
    if own:
        from swa_paged_decode_gb300 import binding as B_
        from swa_paged_decode_gb300 import workloads as W
        s["cache"] = W.PagedCache(s["data"], page, FORMATS[fmt])
        kind = B_.ChunkAttention if case["op"] == "chunk" else B_.AttentionWeights
        s["call"] = kind(T, B, H, width, "cuda", d)
    return s


# ------------------------------------------------------------------ records

def _e4m3(y):
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _bytes(t):
    return t.contiguous().view(torch.uint8).reshape(t.shape[0], -1)


def _pow2_blocks(x, block):
    """Blocks scaled by the smallest power of two that brings them to +-448:
    (codes, scale bytes)."""
    xb = x.reshape(x.shape[0], -1, block)
    frac, e = torch.frexp(xb.abs().amax(-1))
    e = torch.where(frac > 0, e - 9 + (frac > 0.875), torch.zeros_like(e)).clamp(-127, 127)
    return _bytes(_e4m3((xb * torch.exp2(-e.double())[..., None]).float())), (e + 127).to(torch.uint8)


def _encode(fmt, x):
    """[n, dims] in 64 bits -> [n, record] bytes."""
    n = x.shape[0]
    if fmt == "fp8_528_ue8m0":
        return torch.cat(_pow2_blocks(x, 32), 1)
    if fmt == "model1_584":
        codes, scale = _pow2_blocks(x[:, :448], 64)
        return torch.cat([codes, _bytes(x[:, 448:].float().to(torch.bfloat16)), scale, torch.zeros_like(scale[:, :1])], 1)
    if fmt == "nvfp4_288":
        xb = x.reshape(n, 32, 16)
        s8 = _e4m3((xb.abs().amax(-1) / 6.0).float())
        s = s8.double()[..., None]
        y = xb / torch.where(s > 0, s, torch.ones_like(s))
        grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
        code = (y.abs()[..., None] >= (grid[1:] + grid[:-1]) / 2).sum(-1).to(torch.uint8)
        code = (code | ((y < 0).to(torch.uint8) << 3)).reshape(n, 256, 2)
        return torch.cat([code[..., 0] | (code[..., 1] << 4), _bytes(s8)], 1)
    xb = x[:, :DIM].reshape(n, 4, 128)
    s = (xb.abs().amax(-1) / 448.0).float()
    codes = _bytes(_e4m3((xb / torch.where(s > 0, s, torch.ones_like(s)).double()[..., None]).float()))
    parts = [codes, _bytes(s)]
    if fmt == "v32_656":
        parts.append(_bytes(x[:, DIM:].float().to(torch.bfloat16)))
    return torch.cat(parts, 1)


def _values(fmt, rec):
    """[n, record] bytes -> [n, dims] fp32."""
    n = rec.shape[0]

    def part(a, b, dtype):
        return rec[:, a:b].contiguous().view(dtype).float()

    def pow2(a, b):
        return torch.exp2(rec[:, a:b].float() - 127.0)

    if fmt == "nvfp4_288":
        nib = torch.stack([rec[:, :256] & 15, rec[:, :256] >> 4], -1).reshape(n, 512).long()
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=rec.device)
        return (table[nib].reshape(n, 32, 16) * part(256, 288, torch.float8_e4m3fn)[..., None]).reshape(n, 512)
    if fmt == "model1_584":
        c = part(0, 448, torch.float8_e4m3fn).reshape(n, 7, 64) * pow2(576, 583)[..., None]
        return torch.cat([c.reshape(n, 448), part(448, 576, torch.bfloat16)], 1)
    if fmt == "fp8_528_ue8m0":
        return (part(0, 512, torch.float8_e4m3fn).reshape(n, 16, 32) * pow2(512, 528)[..., None]).reshape(n, 512)
    c = (part(0, 512, torch.float8_e4m3fn).reshape(n, 4, 128) * part(512, 528, torch.float32)[..., None]).reshape(n, 512)
    return torch.cat([c, part(528, 656, torch.bfloat16)], 1) if fmt == "v32_656" else c


def _record_views(s):
    """The cache's parts as the values that they hold (no copies)."""
    fmt = s["case"]["fmt"]
    rec = s["data"].view(-1, s["case"]["page"], RECORD[fmt])
    if fmt == "fp8_528_ue8m0":
        return dict(codes=rec[..., :512].view(torch.float8_e4m3fn), scales=rec[..., 512:].view(torch.float8_e8m0fnu))
    if fmt == "model1_584":
        return dict(codes=rec[..., :448].view(torch.float8_e4m3fn), tail=rec[..., 448:576].view(torch.bfloat16),
                    scales=rec[..., 576:583].view(torch.float8_e8m0fnu), unused=rec[..., 583])
    parts = dict(codes=rec[..., :512].view(torch.float8_e4m3fn), scales=rec[..., 512:528].view(torch.float32))
    if fmt == "v32_656":
        parts["tail"] = rec[..., 528:].view(torch.bfloat16)
    return parts


# ------------------------------------------------------------------ plain form

def _rotate(x, table, positions, style):
    """The last 64 dims of x [n, ..., dims] by the rows' angles."""
    cs = table[positions].to(x.dtype)
    while cs.dim() < x.dim():
        cs = cs[:, None]
    c, sn = cs[..., :32], cs[..., 32:]
    r = x[..., -64:]
    if style == NEOX:
        a, b = r[..., :32], r[..., 32:]
        r = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    return torch.cat([x[..., :-64], r], -1)


def _normed(s, x, weight):
    """Rows [T, ..., dims] normed over their first 512 dims and rotated."""
    if weight is not None:
        v = x[..., :DIM]
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
        x = torch.cat([v, x[..., DIM:]], -1)
    if s["table"] is not None:
        x = _rotate(x, s["table"], s["positions"], s["case"]["rope"])
    return x


def _plain_norm(s):
    s["out"].copy_(_normed(s, s["q"].float(), s["q_weight"]))
    keep = s["slots"] >= 0
    # (in 64 bits: a code next to a border falls to the other side of it in 32)
    rows = _encode(s["case"]["fmt"], _normed(s, s["keys"].double(), s["k_weight"])[keep])
    s["data"].view(-1, RECORD[s["case"]["fmt"]])[s["slots"][keep].long()] = rows


def _scores(s):
    """Of every run of query rows: (rows of [T * H], (sequence, values of its
    keys), scaled scores [rows, list length], -inf where a row does not attend)."""
    H, window = s["case"]["H"], s["case"]["window"]
    q = s["q"].float()
    if s["table"] is not None:
        q = _rotate(q, s["table"], s["positions"], s["case"]["rope"])
    q = q.reshape(-1, q.shape[-1])
    t0 = 0
    for b, (n, length) in enumerate(s["sizes"]):
        ids = s["slots"][b, :length].long()
        keep = (ids >= 0) & (ids < s["num_slots"])
        k = _values(s["case"]["fmt"], s["data"].view(-1, RECORD[s["case"]["fmt"]])[ids.clamp(0)])
        j = torch.arange(length, device=ids.device)
        step = max(1, (1 << 29) // (H * length))
        for a in range(0, n, step):
            e = min(n, a + step)
            x = (q[(t0 + a) * H:(t0 + e) * H] @ k.T) * s["scale"]
            p = torch.arange(a, e, device=ids.device).repeat_interleave(H)[:, None] + (length - n)
            seen = keep & (j <= p)
            if window:
                seen = seen & (j > p - window)
            yield slice((t0 + a) * H, (t0 + e) * H), (b, k), x.masked_fill_(~seen, -math.inf)
        t0 += n


def _plain_chunk(s):
    T, H = s["q"].shape[:2]
    out = torch.empty((T * H, DIM), dtype=torch.bfloat16, device="cuda")
    total = torch.empty(T * H, device="cuda")
    sink = None if s["sink"] is None else s["sink"].repeat(T)
    for rows, (_, k), x in _scores(s):
        m = x.amax(-1, keepdim=True)
        m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
        p = x.sub_(m).exp_()
        z = p.sum(-1, keepdim=True)
        lse = (m + z.log())[:, 0]
        o = (p @ k[:, :DIM]) / z.clamp_min(1e-30)
        both = lse
        if s["tail_lse"] is not None:
            tail = s["tail_lse"].view(-1)[rows]
            both = torch.logaddexp(lse, tail)
            o = o * (lse - both).exp()[:, None] + s["tail_out"].view(-1, DIM)[rows].float() * (tail - both).exp()[:, None]
        if sink is not None:
            o = o / (1.0 + (sink[rows] - both).exp())[:, None]
        out[rows], total[rows] = o.to(torch.bfloat16), both
    return dict(out=out.view(T, H, DIM), lse=total.view(T, H))


def _plain_weights(s):
    T = s["q"].shape[0]
    below = s["lse"] if s["sink"] is None else torch.logaddexp(s["lse"], s["sink"])
    below = below.masked_fill(below == -math.inf, math.inf).view(-1)   # a row that attended nothing has no weights
    for b, (_, length) in enumerate(s["sizes"]):
        s["sums"][b, :length] = s["before"][b, :length]
    for rows, (b, _), x in _scores(s):
        s["sums"][b, :x.shape[1]] += (x - below[rows][:, None]).exp_().sum(0)
    return dict(sums=s["sums"])


def _plain_evict(s):
    c = s["case"]
    n, width = s["slots"].shape
    length, j = s["lengths"].long()[:, None], torch.arange(width, device="cuda")[None, :]
    live = j < length
    budget = length.clamp_max(c["budget"])
    first = budget.clamp_max(c["first"])
    last = (budget - first).clamp_max(c["last"])
    # protected entries above all others, entries past the list below all
    rank = torch.where((j < first) | (j >= length - last), torch.full_like(s["scores"], math.inf), s["scores"])
    rank = torch.where(live, rank, torch.full_like(rank, -math.inf))
    order = torch.argsort(rank, dim=1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, j.expand(n, width))
    keep = live & (place < budget)
    for b in range(n):
        kept = keep[b].nonzero()[:, 0]
        gone = (live[b] & ~keep[b]).nonzero()[:, 0]
        s["kept"][b, :len(kept)] = s["slots"][b, kept]
        s["kept_scores"][b, :len(kept)] = s["scores"][b, kept]
        s["freed"][b, :len(gone)] = s["slots"][b, gone]
    s["kept_lengths"].copy_(keep.sum(1))
    s["freed_counts"].copy_((live & ~keep).sum(1))


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "chunk":
            return _plain_chunk(s)
        if op == "weights":
            return _plain_weights(s)
        (_plain_norm if op == "norm" else _plain_evict)(s)
    else:
        from swa_paged_decode_gb300 import binding as B
        if op == "chunk":
            out, lse = s["call"](s["q"], s["cache"], s["slots"], s["lengths"], s["starts"], s["scale"], window=case["window"],
                                 sink=s["sink"], positions=s["positions"], cos_sin=s["table"], rope_style=max(case["rope"], 0),
                                 tail_out=s["tail_out"], tail_lse=s["tail_lse"])
            return dict(out=out, lse=lse)
        if op == "weights":
            s["call"](s["q"], s["cache"], s["slots"], s["lengths"], s["starts"], s["lse"], s["before"], s["sums"], s["scale"],
                      window=case["window"], sink=s["sink"])
            return dict(sums=s["sums"])
        if op == "norm":
            B.dsa_qk_norm(s["q"], s["out"], q_weight=s["q_weight"], keys=s["keys"], key_weight=s["k_weight"], cache=s["cache"],
                          slots=s["slots"], eps=EPS, positions=s["positions"], cos_sin=s["table"], rope_style=max(case["rope"], 0))
        else:
            B.dsa_evict(s["slots"], s["lengths"], s["scores"], case["budget"], s["kept"], s["kept_scores"], s["kept_lengths"],
                        freed=s["freed"], freed_counts=s["freed_counts"], keep_first=case["first"], keep_last=case["last"])
    if op == "norm":
        return dict(q=s["out"], **_record_views(s))
    return {k: s[k] for k in ("kept", "kept_scores", "kept_lengths", "freed", "freed_counts")}


# ------------------------------------------------------------------ cost

def _attended(n, length, window):
    """Sum over n new tokens of the keys that each attends, and the keys that
    any of them does."""
    p0 = length - n
    if not window:
        return sum(range(p0 + 1, length + 1)), length
    return sum(min(p + 1, window) for p in range(p0, length)), min(length, n + window - 1)


def work(case):
    """Inputs once, outputs once; the products of the attention (in 16 bits)."""
    if case["op"] == "evict":
        rng, b = random.Random(case["ragged"]), 0.0
        for _ in range(case["seqs"]):
            n = rng.randint(case["context"] // 2, case["context"])
            b += 8.0 * n + 8.0 * min(n, case["budget"]) + 4.0 * max(0, n - case["budget"]) + 12
        return {"bytes": b, "flops": 0.0}
    fmt = case["fmt"]
    d, rec = dims(fmt), RECORD[fmt]
    if case["op"] == "norm":
        T, H, size = case["T"], case["H"], 4 if case["type"] == "f32" else 2
        b = T * H * d * (size + 2.0) + T * (1.0 - case["pad"]) * (d * size + rec) + 4.0 * T
        return {"bytes": b + (T * (8 + 256) if case["rope"] >= 0 else 0) + (8 * DIM if case["norm"] else 0), "flops": 0.0}
    H, b, f = case["H"], 0.0, 0.0
    chunk = case["op"] == "chunk"
    for n, length in shape(case):
        pairs, keys = _attended(n, length, case["window"])
        f += 2.0 * H * (d + (DIM if chunk else 0)) * pairs
        b += keys * (1.0 - case["invalid"]) * rec + 4.0 * keys + n * H * (2 * d + 4)
        if chunk:
            b += n * H * 2 * DIM + (n * H * (2 * DIM + 4) if case["tail"] else 0) + (n * (8 + 256) if case["rope"] >= 0 else 0)
        else:
            b += 8.0 * length
    return {"bytes": b, "flops": f * (1.0 - case["invalid"])}


# ------------------------------------------------------------------ 64 bits

def _exact_dense(fmt, rec):
    """Records -> values in 64 bits, through tables of the codes' values."""
    def e4m3(codes):
        c = torch.arange(256, device=rec.device, dtype=torch.float64)
        m, e = c % 8, torch.floor(c / 8) % 16
        v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
        return torch.where(c >= 128, -v, v)[codes.long()]

    def bf16(b):
        b = b.long().reshape(b.shape[0], -1, 2)
        return ((b[..., 0] + 256 * b[..., 1]) << 16).to(torch.int32).view(torch.float32).double()

    def spread(v, size):
        return v.repeat_interleave(size, 1)

    if fmt == "nvfp4_288":
        t = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=rec.device) / 2
        nib = torch.stack([rec[:, :256] % 16, rec[:, :256] // 16], -1).flatten(1).long()
        return torch.where(nib >= 8, -t[nib % 8], t[nib % 8]) * spread(e4m3(rec[:, 256:]), 16)
    if fmt == "model1_584":
        return torch.cat([e4m3(rec[:, :448]) * spread(torch.exp2(rec[:, 576:583].double() - 127), 64), bf16(rec[:, 448:576])], 1)
    if fmt == "fp8_528_ue8m0":
        return e4m3(rec[:, :512]) * spread(torch.exp2(rec[:, 512:].double() - 127), 32)
    v = e4m3(rec[:, :512]) * spread(rec[:, 512:528].contiguous().view(torch.float32).double(), 128)
    return torch.cat([v, bf16(rec[:, 528:])], 1) if fmt == "v32_656" else v


def _exact_e4m3(y):
    """Nearest e4m3 value, ties to even, saturating."""
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3.0)
    return (torch.sign(y) * torch.round(a / step) * step).clamp(-448.0, 448.0)


def _exact_parts(fmt, x):
    """The parts of the records of rows x."""
    most, size = {"fp8_528_ue8m0": (DIM, 32), "model1_584": (448, 64)}.get(fmt, (DIM, 128))
    b = x[:, :most].reshape(x.shape[0], -1, size)
    amax = b.abs().amax(-1, keepdim=True)
    if size == 128:
        s = amax / 448.0
        c = _exact_e4m3(torch.where(s > 0, b / s.float().double().clamp_min(1e-300), b))
    else:
        frac, e = torch.frexp(amax)      # amax = frac 2^e, frac in [1/2, 1)
        s = torch.where(frac > 0, torch.exp2((e - 9 + (frac > 0.875).to(e.dtype)).double()), torch.ones_like(frac))
        c = _exact_e4m3(b / s)
    parts = dict(codes=c.flatten(1), scales=s.flatten(1))
    if most < x.shape[1]:
        parts["tail"] = x[:, most:]
    return parts


def _exact_turned(x, s):
    """x [T, m, dims]: each pair as a complex number times e^{i angle}."""
    if s["table"] is None:
        return x
    t = s["table"][s["positions"]].double()
    r, pairs = x[..., -64:], s["case"]["rope"] == GPTJ
    z = torch.complex(r[..., 0::2], r[..., 1::2]) if pairs else torch.complex(r[..., :32].contiguous(), r[..., 32:].contiguous())
    z = z * torch.complex(t[:, :32].contiguous(), t[:, 32:].contiguous())[:, None, :]
    r = torch.view_as_real(z).flatten(-2) if pairs else torch.cat([z.real, z.imag], -1)
    return torch.cat([x[..., :-64], r], -1)


def _exact_norm(s):
    def normed(x, w):
        if w is not None:
            rms = (x[..., :DIM].square().sum(-1, keepdim=True) / DIM + EPS).sqrt()
            x = torch.cat([x[..., :DIM] / rms * w.double(), x[..., DIM:]], -1)
        return _exact_turned(x, s)

    fmt = s["case"]["fmt"]
    keep = s["slots"] >= 0
    parts = _exact_parts(fmt, normed(s["keys"].double()[:, None], s["k_weight"])[:, 0][keep])
    found = dict(q=normed(s["q"].double(), s["q_weight"]))
    for name, like in _record_views(s).items():
        found[name] = None
        if name != "unused":
            whole = like.to(torch.float64)
            flat = whole.reshape(s["data"].numel() // RECORD[fmt], -1)
            flat[s["slots"][keep].long()] = parts[name]
            found[name] = flat.reshape(like.shape)
    return found


def _exact_evict(s):
    c = s["case"]
    found = {k: s[k].cpu().clone() for k in ("kept", "kept_scores", "kept_lengths", "freed", "freed_counts")}
    for b, n in enumerate(s["lengths"].tolist()):
        slots, scores = s["slots"][b, :n].cpu(), s["scores"][b, :n].cpu()
        if n <= c["budget"]:
            kept = torch.arange(n)
        else:
            lo = min(c["first"], c["budget"])
            hi = n - min(c["last"], c["budget"] - lo)
            middle = sorted(range(lo, hi), key=lambda i, v=scores.tolist(): (-v[i], i))[:c["budget"] - lo - (n - hi)]
            kept = torch.tensor(sorted(list(range(lo)) + middle + list(range(hi, n))), dtype=torch.long)
        gone = torch.ones(n, dtype=torch.bool)
        gone[kept] = False
        found["kept"][b, :len(kept)], found["kept_scores"][b, :len(kept)] = slots[kept], scores[kept]
        found["freed"][b, :n - len(kept)] = slots[gone]
        found["kept_lengths"][b], found["freed_counts"][b] = len(kept), n - len(kept)
    found["kept_scores"] = found["kept_scores"].double()
    return found


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "evict":
        return _exact_evict(s)
    T, H = s["q"].shape[:2]
    q = _exact_turned(s["q"].double(), s)
    sink = None if s["sink"] is None else s["sink"].double()[None, :]
    out = torch.zeros((T, H, DIM), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    sums = s["sums"].double().clone() if case["op"] == "weights" else None
    t = 0
    for b, (n, length) in enumerate(s["sizes"]):
        ids = s["slots"][b, :length].long()
        where = ((ids >= 0) & (ids < s["num_slots"])).nonzero()[:, 0]   # list positions of the kept keys
        k = _exact_dense(case["fmt"], s["data"].view(-1, RECORD[case["fmt"]])[ids[where]])
        if sums is not None:
            sums[b, :length] = s["before"][b, :length].double()
        step = max(1, (1 << 27) // (H * max(1, len(k))))
        for a in range(0, n, step):
            e = min(n, a + step)
            x = s["scale"] * (q[t + a:t + e].reshape(-1, q.shape[-1]) @ k.T).view(e - a, H, len(k))
            p = torch.arange(length - n + a, length - n + e, device="cuda")[:, None]
            blind = where[None, :] > p
            if case["window"]:
                blind = blind | (where[None, :] + case["window"] <= p)
            x.masked_fill_(blind[:, None, :], -math.inf)
            if sums is not None:
                below = s["lse"][t + a:t + e].double()
                below = below if sink is None else torch.logaddexp(below, sink)
                below = torch.where(torch.isinf(below), torch.full_like(below, math.inf), below)
                sums[b, where] += (x - below[..., None]).exp().sum((0, 1))
                continue
            lse[t + a:t + e] = torch.logsumexp(x, 2)
            top = lse[t + a:t + e, :, None]
            w = torch.where(torch.isfinite(top), (x - top).exp(), torch.zeros_like(x))
            out[t + a:t + e] = (w.reshape(-1, len(k)) @ k[:, :DIM]).view(e - a, H, DIM)
        t += n
    if sums is not None:
        return dict(sums=sums)
    total = lse
    if case["tail"]:
        total = torch.logaddexp(lse, s["tail_lse"].double())
    below = total if sink is None else torch.logaddexp(total, sink)
    out = (lse - below).exp()[..., None] * out
    if case["tail"]:
        out = out + (s["tail_lse"].double() - below).exp()[..., None] * s["tail_out"].double()
    return dict(out=out, lse=total)
