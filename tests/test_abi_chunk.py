"""dsa_chunk_plan / dsa_chunk_run: exports, planning and refusals before any
launch (no GPU needed: every call below is invalid or empty)."""
import ctypes
import os
import re

import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W

INVALID, UNSUPPORTED, ALIGN, WORKSPACE, PLAN = -1, -2, -3, -4, -7
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dsa_decode.h")


@pytest.fixture(scope="module")
def lib():
    BLD.build()
    return B.load()


def test_every_declared_call_is_bound(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(dsa_chunk_\w+)\s*\(", src))
    assert names == set(B.EXPORTED_CHUNK)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("args,expect", [
    ((-1, 2, 16, 128, 152, 512), INVALID), ((4, -1, 16, 128, 152, 512), INVALID), ((4, 2, 0, 128, 152, 512), INVALID),
    ((4, 2, 16, 0, 152, 512), INVALID), ((4, 2, 16, 128, -1, 512), INVALID), ((4, 2, 16, 128, 152, 513), INVALID),
    ((1 << 20, 2, 1 << 12, 128, 152, 512), UNSUPPORTED), ((4, 1, 16, 2**31 - 1, 152, 512), UNSUPPORTED),
    ((4, 1 << 15, 16, 1 << 15, 152, 512), UNSUPPORTED), ((4, 2**31 - 1, 16, 1, 152, 512), UNSUPPORTED),
])
def test_plan_refusals(lib, args, expect):
    with pytest.raises(B.DsaError) as e:
        B.dsa_chunk_plan(*args)
    assert e.value.status == expect


def test_plan_needs_somewhere_to_put_it(lib):
    ws = ctypes.c_size_t(0)
    assert lib.dsa_chunk_plan(4, 2, 16, 128, 152, 512, None, ctypes.byref(ws)) == INVALID
    assert lib.dsa_chunk_plan(4, 2, 16, 128, 152, 512, ctypes.byref(B.ChunkPlan()), None) == INVALID


@pytest.mark.parametrize("T,S,H,width,sms,d", [(1, 1, 1, 1, 152, 512), (8, 3, 64, 8192, 152, 512), (130, 20, 20, 1500, 152, 576),
                                               (1024, 1, 128, 16384, 148, 512), (3, 9, 16, 300, 1, 512)])
def test_plan_layout(lib, T, S, H, width, sms, d):
    p, nbytes = B.dsa_chunk_plan(T, S, H, width, sms, d)
    assert p.row_tiles == T * H // 128 + min(S, T) and p.seq_halves == -(-width // 128) + 1
    assert 1 <= p.pairs <= max(1, sms // 2)
    keys, parts = 128 * p.seq_halves * S, 2 * p.pairs * 128
    spans = [(0, 256), (p.ws_info_offset, 8 * keys // 32), (p.ws_key_e_offset, 4 * keys), (p.ws_image_offset, 2 * d * keys),
             (p.ws_row_tile_offset, 32 * p.row_tiles), (p.ws_seq_tile_offset, 4 * S), (p.ws_begin_offset, 8 * (p.pairs + 1)),
             (p.ws_tile_offset, 12 * p.row_tiles), (p.ws_part_lse_offset, 4 * parts), (p.ws_part_o_offset, 2048 * parts)]
    for (a, n), (b, _) in zip(spans, spans[1:] + [(nbytes, 0)]):
        assert a % 256 == 0 and a + n <= b
    assert p.workspace_bytes == nbytes and p.wait_budget_cycles == 0


def desc(**kw):
    d = dict(base=0x10000, num_pages=4, page_stride_bytes=64 * 528, page_size=64, format=W.FMT_FP8_528)
    d.update(kw)
    return B.CacheDesc(d["base"], d["num_pages"], d["page_stride_bytes"], d["page_size"], d["format"])


def run(lib, **kw):
    plan, nbytes = B.dsa_chunk_plan(2, 2, 16, 200, 152)
    a = dict(plan=plan, ws=0x100000, nbytes=nbytes, q=0x20000, qt=16 * 512, qh=512, cache=desc(), slots=0x30000, stride=200,
             lengths=0x40000, starts=0x48000, window=0, sink=None, pos=None, table=None, table_rows=0, style=0, scale=0.04,
             tail=None, tail_lse=None, out=0x50000, lse=0x60000)
    a.update(kw)
    ref = lambda x: None if x is None else ctypes.byref(x)
    return lib.dsa_chunk_run(ref(a["plan"]), a["ws"], a["nbytes"], a["q"], a["qt"], a["qh"], ref(a["cache"]), a["slots"], a["stride"],
                             a["lengths"], a["starts"], a["window"], a["sink"], a["pos"], a["table"], a["table_rows"], a["style"],
                             a["scale"], a["tail"], a["tail_lse"], a["out"], a["lse"], None)


@pytest.mark.parametrize("T,S", [(0, 3), (5, 0)])
def test_nothing_to_do(lib, T, S):
    p, nbytes = B.dsa_chunk_plan(T, S, 16, 128, 152)
    assert nbytes == 0
    assert run(lib, plan=p, q=None, ws=None) == 0


@pytest.mark.parametrize("kw,expect", [
    (dict(plan=None), PLAN), (dict(plan=B.ChunkPlan()), PLAN), (dict(q=None), INVALID), (dict(slots=None), INVALID),
    (dict(lengths=None), INVALID), (dict(starts=None), INVALID), (dict(out=None), INVALID), (dict(lse=None), INVALID),
    (dict(cache=None), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(style=2), INVALID),
    (dict(window=-1), INVALID), (dict(stride=199), INVALID), (dict(qh=504), INVALID), (dict(qt=15 * 512 + 504), INVALID),
    (dict(pos=0x70000), INVALID), (dict(table=0x70000, table_rows=1), INVALID), (dict(pos=0x70000, table=0x80000, table_rows=0), INVALID),
    (dict(tail=0x90000), INVALID), (dict(tail_lse=0x90000), INVALID), (dict(q=0x20008), ALIGN), (dict(qt=16 * 512 + 4), ALIGN),
    (dict(qh=516, qt=16 * 516), ALIGN), (dict(out=0x50008), ALIGN), (dict(lse=0x60002), ALIGN), (dict(slots=0x30001), ALIGN),
    (dict(lengths=0x40002), ALIGN), (dict(starts=0x48002), ALIGN), (dict(sink=0x70002), ALIGN),
    (dict(pos=0x70004, table=0x80000, table_rows=4), ALIGN), (dict(pos=0x70000, table=0x80008, table_rows=4), ALIGN),
    (dict(tail=0x90008, tail_lse=0xA0000), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=0x100080), WORKSPACE),
    (dict(nbytes=1000), WORKSPACE), (dict(cache=desc(base=None)), INVALID), (dict(cache=desc(format=9)), UNSUPPORTED),
    (dict(cache=desc(page_size=65)), INVALID), (dict(cache=desc(format=W.FMT_V32_656, page_stride_bytes=64 * 656)), UNSUPPORTED),
])
def test_run_refusals(lib, kw, expect):
    assert run(lib, **kw) == expect


def test_v32_plan_takes_v32_records_and_no_table(lib):
    plan, nbytes = B.dsa_chunk_plan(2, 2, 16, 200, 152, 576)
    v32 = desc(format=W.FMT_V32_656, page_stride_bytes=64 * 656)
    kw = dict(plan=plan, nbytes=nbytes, qt=16 * 576, qh=576)
    assert run(lib, cache=desc(), **kw) == UNSUPPORTED
    assert run(lib, cache=v32, pos=0x70000, table=0x80000, table_rows=4, **kw) == UNSUPPORTED


def test_wait_budget_knob(lib, monkeypatch):
    monkeypatch.setenv("DSA_DECODE_WAIT_BUDGET", "7")
    assert B.dsa_chunk_plan(2, 2, 16, 200, 152)[0].wait_budget_cycles == 7


def test_binding_refuses_host_tensors(lib):
    plan, nbytes = B.dsa_chunk_plan(2, 1, 16, 200, 152)
    c = W.PagedCache(torch.zeros((4, 64 * 528), dtype=torch.uint8), 64, W.FMT_FP8_528)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)
    with pytest.raises(B.DsaError):
        B.dsa_chunk_run(plan, torch.zeros(nbytes, dtype=torch.uint8), torch.zeros((2, 16, 512), dtype=torch.bfloat16), c,
                        i32(1, 200), i32(1), i32(2), 0, None, None, None, 0, 0.04, None, None,
                        torch.zeros((2, 16, 512), dtype=torch.bfloat16), torch.zeros((2, 16)))
