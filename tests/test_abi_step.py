"""dsa_qk_norm and dsa_evict: exports and refusals before any launch (no GPU
needed: every call below is invalid or empty)."""
import ctypes
import os
import re

import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W

INVALID, UNSUPPORTED, ALIGN = -1, -2, -3
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dsa_decode.h")


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return B.load()


def test_every_declared_call_is_bound(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(dsa_(?:qk|evict)\w*)\s*\(", src))
    assert names == set(B.EXPORTED_STEP)
    for n in names:
        assert hasattr(lib, n), n


def desc(**kw):
    d = dict(base=0x10000, num_pages=4, page_stride_bytes=64 * 528, page_size=64, format=W.FMT_FP8_528)
    d.update(kw)
    return B.CacheDesc(d["base"], d["num_pages"], d["page_stride_bytes"], d["page_size"], d["format"])


def norm(lib, **kw):
    a = dict(T=3, H=16, d=512, type=0, q=0x20000, qt=16 * 512, qh=512, w=0x30000, wh=0, out=0x40000, ot=16 * 512, oh=512,
             keys=0x50000, ks=512, kw=0x60000, cache=desc(), slots=0x70000, eps=1e-6, pos=0x80000, table=0x90000, rows=8, style=0,
             status=None)
    a.update(kw)
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    return lib.dsa_qk_norm(a["T"], a["H"], a["d"], a["type"], a["q"], a["qt"], a["qh"], a["w"], a["wh"], a["out"], a["ot"], a["oh"],
                           a["keys"], a["ks"], a["kw"], c, a["slots"], a["eps"], a["pos"], a["table"], a["rows"], a["style"],
                           a["status"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(d=513), INVALID), (dict(type=3), UNSUPPORTED), (dict(type=-1), UNSUPPORTED),
    (dict(T=1 << 20, H=1 << 12), UNSUPPORTED), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(style=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID), (dict(pos=None), INVALID), (dict(table=None), INVALID),
    (dict(rows=0), INVALID), (dict(qh=504), INVALID), (dict(qt=15 * 512), INVALID), (dict(oh=504), INVALID), (dict(ot=15 * 512), INVALID),
    (dict(ks=504), INVALID), (dict(wh=508), INVALID), (dict(keys=None), INVALID), (dict(slots=None), INVALID), (dict(cache=None), INVALID),
    (dict(cache=desc(format=9)), UNSUPPORTED), (dict(cache=desc(format=W.FMT_V32_656, page_stride_bytes=64 * 656)), UNSUPPORTED),
    (dict(d=576, qt=16 * 576, qh=576, ot=16 * 576, oh=576, ks=576), UNSUPPORTED), (dict(out=0x20000, type=2), INVALID),
    (dict(out=0x20000, qh=520, qt=16 * 520), INVALID), (dict(q=0x20008), ALIGN), (dict(qh=516, qt=16 * 516), ALIGN),
    (dict(qt=16 * 512 + 4), ALIGN), (dict(out=0x40008), ALIGN), (dict(oh=516, ot=16 * 516), ALIGN), (dict(w=0x30004), ALIGN),
    (dict(wh=514), ALIGN), (dict(keys=0x50008), ALIGN), (dict(ks=516), ALIGN), (dict(slots=0x70002), ALIGN), (dict(kw=0x60004), ALIGN),
    (dict(pos=0x80004), ALIGN), (dict(table=0x90008), ALIGN), (dict(status=0x90002), ALIGN),
])
def test_norm_refusals(lib, kw, expect):
    assert norm(lib, **kw) == expect


def test_norm_of_no_tokens(lib):
    assert norm(lib, T=0, q=None, out=None, keys=None, slots=None, pos=None) == 0


def evict(lib, **kw):
    a = dict(n=2, width=100, slots=0x10000, ss=100, lengths=0x20000, scores=0x30000, cs=100, budget=30, first=0, last=0, kept=0x40000,
             ks=30, kscores=0x50000, kcs=30, klen=0x60000, freed=0x70000, fs=70, counts=0x80000)
    a.update(kw)
    return lib.dsa_evict(a["n"], a["width"], a["slots"], a["ss"], a["lengths"], a["scores"], a["cs"], a["budget"], a["first"], a["last"],
                         a["kept"], a["ks"], a["kscores"], a["kcs"], a["klen"], a["freed"], a["fs"], a["counts"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), INVALID), (dict(width=0), INVALID), (dict(budget=0), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(n=2**31 - 1), UNSUPPORTED), (dict(width=2**31 - 1, ss=2**31, cs=2**31, fs=2**31), UNSUPPORTED), (dict(slots=None), INVALID),
    (dict(lengths=None), INVALID), (dict(scores=None), INVALID), (dict(kept=None), INVALID), (dict(kscores=None), INVALID),
    (dict(klen=None), INVALID), (dict(freed=None), INVALID), (dict(counts=None), INVALID), (dict(ss=99), INVALID), (dict(cs=99), INVALID),
    (dict(ks=29), INVALID), (dict(kcs=29), INVALID), (dict(fs=69), INVALID), (dict(kept=0x10000), INVALID), (dict(kscores=0x30000), INVALID),
    (dict(freed=0x10000), INVALID), (dict(slots=0x10002), ALIGN), (dict(lengths=0x20001), ALIGN), (dict(scores=0x30002), ALIGN),
    (dict(kept=0x40002), ALIGN), (dict(kscores=0x50001), ALIGN), (dict(klen=0x60002), ALIGN), (dict(freed=0x70001), ALIGN),
    (dict(counts=0x80002), ALIGN),
])
def test_evict_refusals(lib, kw, expect):
    assert evict(lib, **kw) == expect


@pytest.mark.parametrize("kw", [dict(klen=0x20000), dict(counts=0x20000), dict(counts=0x60000), dict(freed=0x40000)])
def test_evict_refuses_outputs_in_place_of_lengths_or_one_another(lib, kw):
    """Every CTA of a list reads its length while the first one writes the new one."""
    assert evict(lib, **kw) == INVALID


def test_evict_of_no_lists(lib):
    assert evict(lib, n=0, slots=None) == 0


def test_binding_refuses_host_tensors(lib):
    z = torch.zeros((2, 16, 512), dtype=torch.bfloat16)
    with pytest.raises(B.DsaError):
        B.dsa_qk_norm(z, z)
    i = torch.zeros((2, 8), dtype=torch.int32)
    with pytest.raises(B.DsaError):
        B.dsa_evict(i, i[:, 0].contiguous(), torch.zeros((2, 8)), 4, i.clone(), torch.zeros((2, 8)), i[:, 0].contiguous())
