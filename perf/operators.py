"""The measured cases of the cache and shared-prefix operators.

Three operators that sit around the paged decode:

  * cache write: rows of keys (as the model's projection leaves them) are
    optionally RMS-normed and rotated, quantized into one of the five record
    formats and stored at the paged slots of a cache;
  * cache read: records named by slot ids come back as dense rows;
  * shared-prefix attention: every token of a decode batch attends to one
    common list of records (a system prompt, a document), gathered and
    dequantized once for all of them; the result is merged with the state of
    the token's own list when one is given.

``run`` computes a case in its plain form (elementary torch operations, 32
bits or more) or, with ``own`` set, by the package's calls.
"""
import math

import torch

own = False

DIM = 512
ROPE_ROWS = 131072
NEOX, GPTJ = 0, 1
FORMATS = {"fp8_528": 0, "nvfp4_288": 1, "fp8_528_ue8m0": 2, "model1_584": 3, "v32_656": 4}
RECORD = {"fp8_528": 528, "nvfp4_288": 288, "fp8_528_ue8m0": 528, "model1_584": 584, "v32_656": 656}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def dims(fmt):
    """Dims of a key: V3.2 records carry 64 more than the value."""
    return 576 if fmt == "v32_656" else DIM


def listed():
    return [
        # one decode step of 32 requests appends its keys (latency counts)
        dict(name="write_step_fp8", op="write", fmt="fp8_528", n=32, slots=4096, page=64, type="bf16", norm=False, rope=NEOX, pad=0.1),
        # a chunk of a prefill, an odd count, fp32 rows from an unfused projection
        dict(name="write_chunk_ue8m0", op="write", fmt="fp8_528_ue8m0", n=4099, slots=8192, page=64, type="f32", norm=False, rope=GPTJ, pad=0.0),
        # prefill of a large batch: norm, rotation and quantization in one pass
        dict(name="write_prefill_model1", op="write", fmt="model1_584", n=65536, slots=65536, page=64, type="bf16", norm=True, rope=GPTJ, pad=0.0),
        # a chunk quantized to the extra cache and read back for the dense prefill attention
        dict(name="write_read_nvfp4", op="write_read", fmt="nvfp4_288", n=8192, slots=8192, page=256, type="bf16", norm=True, rope=-1, pad=0.0),
        # the sliding-window rows of a few tokens, for a check in fp32
        dict(name="read_window_fp8", op="read", fmt="fp8_528", n=640, slots=65536, page=64, type="f32", pad=0.05),
        # a long cached context read back for a dense prefill
        dict(name="read_context_nvfp4", op="read", fmt="nvfp4_288", n=131072, slots=1 << 18, page=256, type="bf16", pad=0.0),
        # two requests behind a short system prompt (latency counts)
        dict(name="prefix_small", op="prefix", fmt="fp8_528", T=2, H=16, P=512, page=64, rope=-1, sink=False, tail=False, invalid=0.0, short=0),
        # a chat batch behind an 8K prompt, the extra cache's records
        dict(name="prefix_chat_nvfp4", op="prefix", fmt="nvfp4_288", T=8, H=64, P=8192, page=256, rope=NEOX, sink=True, tail=False, invalid=0.0, short=0),
        # a batch behind a 4K document, merged with each token's own window
        dict(name="prefix_merge_ue8m0", op="prefix", fmt="fp8_528_ue8m0", T=32, H=64, P=4096, page=64, rope=GPTJ, sink=True, tail=True, invalid=0.0, short=0),
        # odd counts of everything: tokens, heads, length; unused slots in the list
        dict(name="prefix_ragged_v32", op="prefix", fmt="v32_656", T=13, H=20, P=1500, page=64, rope=-1, sink=True, tail=True, invalid=0.03, short=77),
        # few requests behind a very long document
        dict(name="prefix_long_model1", op="prefix", fmt="model1_584", T=4, H=64, P=65536, page=64, rope=NEOX, sink=True, tail=True, invalid=0.0, short=0),
        # a full decode batch of the widest layer behind a 16K document
        dict(name="prefix_batch_fp8", op="prefix", fmt="fp8_528", T=128, H=128, P=16384, page=64, rope=NEOX, sink=True, tail=True, invalid=0.0, short=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    fmt = rng.choice(list(FORMATS))
    page = rng.choice([16, 64, 128, 256])
    op = rng.choice(["write", "write_read", "read", "prefix", "prefix", "prefix"])
    if op != "prefix":
        n = _log(rng, 1, 65536)
        slots = -(-max(n + rng.randrange(0, n + 1), page) // page) * page
        case = dict(op=op, fmt=fmt, n=n, slots=slots, page=page, type=rng.choice(list(TYPES)), pad=rng.choice([0.0, 0.0, 0.1]))
        if op != "read":
            case.update(norm=rng.random() < 0.5, rope=rng.choice([-1, NEOX, GPTJ]))
            if op == "write" and fmt == "nvfp4_288":
                case["op"] = "write_read"   # 4-bit codes are compared as the values they stand for
        return case
    while True:
        T, H, P = _log(rng, 1, 256), rng.choice([8, 16, 20, 32, 40, 64, 96, 128]), _log(rng, 256, 65536)
        if T * H * P <= 128 * 128 * 16384:
            break
    return dict(op="prefix", fmt=fmt, T=T, H=H, P=P, page=page, rope=-1 if fmt == "v32_656" else rng.choice([-1, NEOX, GPTJ]),
                sink=rng.random() < 0.5, tail=rng.random() < 0.5, invalid=rng.choice([0.0, 0.0, 0.05]),
                short=rng.choice([0, rng.randrange(0, P // 4)]))


# ------------------------------------------------------------------ inputs

def _table(device):
    """[rows, 64] rows of 32 cosines and 32 sines, angles in 64 bits."""
    w = 10000.0 ** (-torch.arange(32, dtype=torch.float64, device=device) / 32.0)
    a = torch.arange(ROPE_ROWS, dtype=torch.float64, device=device)[:, None] * w
    return torch.cat([a.cos(), a.sin()], 1).float()


def _paged_list(n, num_slots, page, gen, device):
    """n distinct slots as an allocator hands them out: whole pages in any
    order, their slots in sequence."""
    pages = torch.randperm(num_slots // page, generator=gen, device=device)[: -(-n // page)]
    ids = pages[:, None] * page + torch.arange(page, device=device)
    return ids.reshape(-1)[:n].to(torch.int32)


def _drop(ids, share, gen):
    if share > 0:
        ids = torch.where(torch.rand(ids.shape, generator=gen, device=ids.device) < share, torch.full_like(ids, -1), ids)
    return ids


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    fmt, page = case["fmt"], case["page"]
    prefix = case["op"] == "prefix"
    n = case["P"] if prefix else case["n"]
    num_slots = -(-n // page) * page + 4 * page if prefix else case["slots"]
    pages = num_slots // page
    data = torch.zeros((pages, page * RECORD[fmt]), dtype=torch.uint8, device=dev)
    s = dict(case=case, fmt=fmt, page=page, data=data, num_slots=num_slots)
    if case["op"] in ("read", "prefix"):   # the cache holds quantized N(0, 1) rows
        rec = data.view(num_slots, RECORD[fmt])
        for a in range(0, num_slots, 1 << 16):
            b = min(num_slots, a + (1 << 16))
            rec[a:b] = _encode(fmt, torch.randn((b - a, dims(fmt)), generator=g, device=dev, dtype=torch.float32).double())
    ids = _paged_list(n, num_slots, page, g, dev)
    s["slots"] = _drop(ids, case["invalid"] if prefix else case["pad"], g).contiguous()
    if prefix:
        T, H = case["T"], case["H"]
        s["length"] = torch.tensor([n - case["short"]], dtype=torch.int32, device=dev)
        s["q"] = torch.randn((T, H, dims(fmt)), generator=g, device=dev).to(torch.bfloat16)
        s["scale"] = dims(fmt) ** -0.5
        s["sink"] = torch.randn((H,), generator=g, device=dev) if case["sink"] else None
        s["tail_out"] = s["tail_lse"] = None
        if case["tail"]:   # the state that the decode of the token's own list left
            s["tail_out"] = (0.2 * torch.randn((T, H, DIM), generator=g, device=dev)).to(torch.bfloat16)
            s["tail_lse"] = 5.0 + torch.randn((T, H), generator=g, device=dev)
        rows = T
    else:
        s["rows"] = None
        if case["op"] != "read":
            s["rows"] = torch.randn((n, dims(fmt)), generator=g, device=dev).to(TYPES[case["type"]])
        if case["op"] != "write":
            s["dense"] = torch.empty((n, dims(fmt)), dtype=TYPES[case["type"]], device=dev)
        s["norm"] = 1.0 + 0.1 * torch.randn((DIM,), generator=g, device=dev) if case.get("norm") else None
        rows = n
    s["positions"] = s["table"] = None
    if case.get("rope", -1) >= 0:
        s["positions"] = torch.randint(0, ROPE_ROWS, (rows,), generator=g, device=dev)
        s["table"] = _table(dev)
    if own:
        from swa_paged_decode_gb300 import binding as B
        from swa_paged_decode_gb300 import workloads as W
        s["cache"] = W.PagedCache(data, page, FORMATS[fmt])
        if prefix:
            s["attn"] = B.PrefixAttention(case["T"], case["H"], n, device=dev, d_qk=dims(fmt))
    return s


# ------------------------------------------------------------------ plain form

def _e4m3(y):
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _bytes(t):
    return t.contiguous().view(torch.uint8).reshape(t.shape[0], -1)


def _pow2_blocks(x, block):
    """Blocks scaled by the smallest power of two that brings them to +-448:
    (codes, scale bytes)."""
    xb = x.reshape(x.shape[0], -1, block)
    amax = xb.abs().amax(-1)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448.0)), torch.zeros_like(amax)).clamp(-127, 127)
    return _bytes(_e4m3((xb / torch.exp2(e)[..., None]).float())), (e + 127).to(torch.uint8)


def _encode(fmt, x):
    """[n, dims] in 64 bits -> [n, record] bytes."""
    n = x.shape[0]
    if fmt == "fp8_528_ue8m0":
        return torch.cat(_pow2_blocks(x, 32), 1)
    if fmt == "model1_584":
        codes, scale = _pow2_blocks(x[:, :448], 64)
        tail = _bytes(x[:, 448:].float().to(torch.bfloat16))
        return torch.cat([codes, tail, scale, torch.zeros((n, 1), dtype=torch.uint8, device=x.device)], 1)
    if fmt == "nvfp4_288":
        xb = x.reshape(n, 32, 16)
        s8 = _e4m3((xb.abs().amax(-1) / 6.0).float())
        s = s8.double()[..., None]
        y = torch.where(s > 0, xb / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(xb))
        a = y.abs()
        code = sum(((a > b) if strict else (a >= b)).to(torch.uint8) for b, strict in
                   ((0.25, True), (0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)))
        code = code | (((y < 0) & (code > 0)).to(torch.uint8) << 3)
        code = code.reshape(n, 256, 2)
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


EPS = 1e-6


def _source(s):
    """The rows to be quantized, in 64 bits."""
    x = s["rows"].double()
    if s["norm"] is not None:
        v = x[:, :DIM]
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * s["norm"].double()
        x = torch.cat([v, x[:, DIM:]], 1)
    if s["table"] is not None:
        x = _rotate(x, s["table"], s["positions"], s["case"]["rope"])
    return x


def _kept(s, ids):
    return (ids >= 0) & (ids < s["num_slots"])


def _record_views(s):
    """The cache's parts as the values that they hold (no copies)."""
    fmt = s["fmt"]
    rec = s["data"].view(-1, s["page"], RECORD[fmt])
    if fmt == "fp8_528_ue8m0":
        return dict(codes=rec[..., :512].view(torch.float8_e4m3fn), scales=rec[..., 512:].view(torch.float8_e8m0fnu))
    if fmt == "model1_584":
        return dict(codes=rec[..., :448].view(torch.float8_e4m3fn), tail=rec[..., 448:576].view(torch.bfloat16),
                    scales=rec[..., 576:583].view(torch.float8_e8m0fnu), unused=rec[..., 583])
    parts = dict(codes=rec[..., :512].view(torch.float8_e4m3fn), scales=rec[..., 512:528].view(torch.float32))
    if fmt == "v32_656":
        parts["tail"] = rec[..., 528:].view(torch.bfloat16)
    return parts


def _plain_write(s):
    ids = s["slots"].long()
    keep = _kept(s, ids)
    s["data"].view(-1, RECORD[s["fmt"]])[ids[keep]] = _encode(s["fmt"], _source(s)[keep])


def _plain_read(s):
    ids = s["slots"].long()
    keep = _kept(s, ids)
    v = _values(s["fmt"], s["data"].view(-1, RECORD[s["fmt"]])[torch.where(keep, ids, torch.zeros_like(ids))])
    return torch.where(keep[:, None], v, torch.zeros_like(v)).to(s["dense"].dtype)


def _plain_prefix(s):
    T, H = s["q"].shape[:2]
    ids = s["slots"].long()
    keep = _kept(s, ids) & (torch.arange(len(ids), device=ids.device) < s["length"])
    k = _values(s["fmt"], s["data"].view(-1, RECORD[s["fmt"]])[torch.where(keep, ids, torch.zeros_like(ids))])
    q = s["q"].float()
    if s["table"] is not None:
        q = _rotate(q, s["table"], s["positions"], s["case"]["rope"])
    x = (q.reshape(T * H, -1) @ k.T) * s["scale"]
    x = x.masked_fill_(~keep[None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    lse = (m + z.log()).reshape(T, H)
    o = (p @ k[:, :DIM]).reshape(T, H, DIM) / z.reshape(T, H, 1).clamp_min(1e-30)
    tail = s["tail_lse"]
    both = lse if tail is None else torch.logaddexp(lse, tail)
    w = (lse - both).exp()[..., None]
    o = o * w
    if tail is not None:
        o = o + s["tail_out"].float() * (tail - both).exp()[..., None]
    if s["sink"] is not None:
        o = o / (1.0 + (s["sink"][None, :] - both).exp())[..., None]
    return o.to(torch.bfloat16), both


def run(s):
    op = s["case"]["op"]
    if own:
        from swa_paged_decode_gb300 import binding as B
        if op == "prefix":
            out, lse = s["attn"](s["q"], s["cache"], s["slots"], s["length"], s["scale"], sink=s["sink"], positions=s["positions"],
                                 cos_sin=s["table"], rope_style=max(s["case"]["rope"], 0), tail_out=s["tail_out"], tail_lse=s["tail_lse"])
            return dict(out=out, lse=lse)
        if op != "read":
            B.dsa_cache_write(s["cache"], s["slots"], s["rows"], norm_weight=s["norm"], norm_eps=EPS, positions=s["positions"],
                              cos_sin=s["table"], rope_style=max(s["case"]["rope"], 0))
        if op != "write":
            B.dsa_cache_read(s["cache"], s["slots"], s["dense"])
    else:
        if op == "prefix":
            out, lse = _plain_prefix(s)
            return dict(out=out, lse=lse)
        if op != "read":
            _plain_write(s)
        if op != "write":
            s["dense"] = _plain_read(s)
    return _record_views(s) if op == "write" else dict(dense=s["dense"])


# ------------------------------------------------------------------ cost

def work(case):
    """Inputs once, outputs once; the products of the attention (in 16 bits)."""
    fmt = case["fmt"]
    d, rec = dims(fmt), RECORD[fmt]
    if case["op"] == "prefix":
        T, H = case["T"], case["H"]
        n = (case["P"] - case["short"]) * (1.0 - case["invalid"])
        b = T * H * (2 * d + 2 * DIM + 4) + n * (rec + 4)
        if case["tail"]:
            b += T * H * (2 * DIM + 4)
        if case["rope"] >= 0:
            b += T * (8 + 256)
        return {"bytes": b, "flops": 2.0 * T * H * n * (d + DIM)}
    n = case["n"] * (1.0 - case["pad"])
    size = 4 if case["type"] == "f32" else 2
    b = 4.0 * case["n"]
    if case["op"] != "read":
        b += n * (d * size + rec) + (n * (8 + 256) if case["rope"] >= 0 else 0) + (4 * DIM if case["norm"] else 0)
    if case["op"] != "write":
        b += n * rec + case["n"] * d * size
    return {"bytes": b, "flops": 0.0}


# ------------------------------------------------------------------ 64 bits

def _exact_e4m3(y):
    """Nearest e4m3 value, ties to even, saturating."""
    a = y.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3.0)
    return (torch.sign(y) * torch.round(a / step) * step).clamp(-448.0, 448.0)


def _exact_e2m1(y):
    a = y.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(a.dtype)
    return torch.sign(y) * (torch.round(a / step) * step).clamp_max(6.0)


def _exact_parts(fmt, x):
    """(parts of the records, the values that they stand for) of rows x."""
    def blocks(v, size):
        return v.reshape(v.shape[0], -1, size)

    if fmt == "nvfp4_288":
        b = blocks(x, 16)
        s = _exact_e4m3(b.abs().amax(-1, keepdim=True) / 6.0)
        y = _exact_e2m1(torch.where(s > 0, b / s.clamp_min(1e-300), torch.zeros_like(b)))
        return {}, (y * s).flatten(1)
    if fmt in ("fp8_528", "v32_656"):
        b = blocks(x[:, :DIM], 128)
        s = b.abs().amax(-1, keepdim=True) / 448.0
        c = _exact_e4m3(torch.where(s > 0, b / s.float().double().clamp_min(1e-300), b))
        parts, v = dict(codes=c.flatten(1), scales=s.flatten(1)), (c * s).flatten(1)
        if fmt == "v32_656":
            parts["tail"] = x[:, DIM:]
            v = torch.cat([v, x[:, DIM:]], 1)
        return parts, v
    size, most = (32, DIM) if fmt == "fp8_528_ue8m0" else (64, 448)
    b = blocks(x[:, :most], size)
    frac, e = torch.frexp(b.abs().amax(-1, keepdim=True))      # amax = frac 2^e, frac in [1/2, 1)
    s = torch.where(frac > 0, torch.exp2((e - 9 + (frac > 0.875).to(e.dtype)).double()), torch.ones_like(frac))
    c = _exact_e4m3(b / s)
    parts, v = dict(codes=c.flatten(1), scales=s.flatten(1)), (c * s).flatten(1)
    if fmt == "model1_584":
        parts["tail"] = x[:, most:]
        v = torch.cat([v, x[:, most:]], 1)
    return parts, v


def _exact_rotated(x, s):
    """x [n, m, dims]: each pair as a complex number times e^{i angle}."""
    if s["table"] is None:
        return x
    t = s["table"][s["positions"]].double()
    turn = torch.complex(t[:, :32], t[:, 32:])[:, None, :]
    r, pairs = x[..., -64:], s["case"]["rope"] == GPTJ
    z = torch.complex(r[..., 0::2], r[..., 1::2]) if pairs else torch.complex(r[..., :32], r[..., 32:])
    z = z * turn
    r = torch.view_as_real(z).flatten(-2) if pairs else torch.cat([z.real, z.imag], -1)
    return torch.cat([x[..., :-64], r], -1)


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


def exact(case, seed):
    s = prepare(case, seed)
    fmt, ids = case["fmt"], s["slots"].long()
    keep = (ids >= 0) & (ids < s["num_slots"])
    if case["op"] in ("write", "write_read"):
        x = s["rows"].double()
        if s["norm"] is not None:
            rms = (x[:, :DIM].square().sum(1, keepdim=True) / DIM + EPS).sqrt()
            x = torch.cat([x[:, :DIM] / rms * s["norm"].double(), x[:, DIM:]], 1)
        x = _exact_rotated(x[:, None], s)[:, 0]
        parts, v = _exact_parts(fmt, x[keep])
        if case["op"] == "write_read":
            dense = torch.zeros((len(ids), dims(fmt)), dtype=torch.float64, device=x.device)
            dense[keep] = v
            return dict(dense=dense)
        found = {}
        for name, like in _record_views(s).items():
            whole = like.to(torch.float64) if name != "unused" else None
            if whole is not None:
                flat = whole.reshape(s["num_slots"], -1)
                flat[ids[keep]] = parts[name]
                whole = flat.reshape(like.shape)
            found[name] = whole
        return found
    rec = s["data"].view(-1, RECORD[fmt])
    if case["op"] == "read":
        dense = torch.zeros((len(ids), dims(fmt)), dtype=torch.float64, device=rec.device)
        dense[keep] = _exact_dense(fmt, rec[ids[keep]])
        return dict(dense=dense)
    keep[int(s["length"]):] = False
    k = _exact_dense(fmt, rec[ids[keep]])
    T, H = case["T"], case["H"]
    q = _exact_rotated(s["q"].double(), s).reshape(T * H, -1)
    out = torch.empty((T * H, DIM), dtype=torch.float64, device=k.device)
    lse = torch.empty((T * H,), dtype=torch.float64, device=k.device)
    step = max(1, (1 << 27) // max(1, len(k)))
    for a in range(0, T * H, step):
        x = s["scale"] * (q[a:a + step] @ k.T)
        lse[a:a + step] = torch.logsumexp(x, 1)
        out[a:a + step] = torch.softmax(x, 1) @ k[:, :DIM]
    parts = [(lse.reshape(T, H), out.reshape(T, H, DIM))]
    if case["tail"]:
        parts.append((s["tail_lse"].double(), s["tail_out"].double()))
    total = torch.logsumexp(torch.stack([p[0] for p in parts]), 0)
    below = total if s["sink"] is None else torch.logaddexp(total, s["sink"].double()[None, :])
    return dict(out=sum((l - below).exp()[..., None] * o for l, o in parts), lse=total)
