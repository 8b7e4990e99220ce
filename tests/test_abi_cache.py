"""dsa_cache_write / dsa_cache_read: the library exports them and refuses bad
arguments before any launch (no GPU needed: every call below is invalid)."""
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
    names = set(re.findall(r"\b(dsa_cache_\w+)\s*\(", src))
    assert names == set(B.EXPORTED_CACHE)
    for n in names:
        assert hasattr(lib, n), n


def desc(**kw):
    d = dict(base=0x10000, num_pages=4, page_stride_bytes=64 * 528, page_size=64, format=W.FMT_FP8_528)
    d.update(kw)
    return B.CacheDesc(d["base"], d["num_pages"], d["page_stride_bytes"], d["page_size"], d["format"])


WRITE = dict(cache=desc(), slots=0x20000, n=8, rows=0x30000, stride=512, type=0, norm=None, eps=0.0,
             pos=None, table=None, table_rows=0, style=0, status=None)


def write(lib, **kw):
    a = dict(WRITE, **kw)
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    return lib.dsa_cache_write(c, a["slots"], a["n"], a["rows"], a["stride"], a["type"], a["norm"],
                               a["eps"], a["pos"], a["table"], a["table_rows"], a["style"],
                               a["status"], None)


def read(lib, **kw):
    a = dict(WRITE, **kw)
    c = None if a["cache"] is None else ctypes.byref(a["cache"])
    return lib.dsa_cache_read(c, a["slots"], a["n"], a["rows"], a["stride"], a["type"], None)


SHARED = [
    (dict(cache=None), INVALID), (dict(cache=desc(base=None)), INVALID),
    (dict(cache=desc(format=5)), UNSUPPORTED), (dict(cache=desc(format=-1)), UNSUPPORTED),
    (dict(cache=desc(num_pages=0)), INVALID), (dict(cache=desc(page_size=48)), INVALID),
    (dict(cache=desc(page_size=0)), INVALID), (dict(cache=desc(page_stride_bytes=64 * 528 - 16)), INVALID),
    (dict(cache=desc(num_pages=1 << 26)), UNSUPPORTED), (dict(cache=desc(base=0x10008)), ALIGN),
    (dict(cache=desc(page_stride_bytes=64 * 528 + 8)), ALIGN),
    (dict(n=-1), INVALID), (dict(slots=None), INVALID), (dict(rows=None), INVALID),
    (dict(type=3), UNSUPPORTED), (dict(type=-1), UNSUPPORTED), (dict(stride=511), INVALID),
    (dict(cache=desc(format=W.FMT_V32_656, page_stride_bytes=64 * 656), stride=512), INVALID),
    (dict(rows=0x30008), ALIGN), (dict(stride=516), ALIGN), (dict(type=2, stride=514), ALIGN),
    (dict(slots=0x20002), ALIGN), (dict(n=1 << 40), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", SHARED)
def test_refusals_of_both(lib, kw, expect):
    assert write(lib, **kw) == expect
    assert read(lib, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(style=2), INVALID), (dict(pos=0x40000), INVALID), (dict(table=0x50000, table_rows=4), INVALID),
    (dict(pos=0x40000, table=0x50000, table_rows=0), INVALID),
    (dict(pos=0x40004, table=0x50000, table_rows=4), ALIGN), (dict(pos=0x40000, table=0x50008, table_rows=4), ALIGN),
    (dict(norm=0x60004), ALIGN), (dict(norm=0x60000, eps=-1.0), INVALID),
    (dict(norm=0x60000, eps=float("nan")), INVALID), (dict(norm=0x60000, eps=float("inf")), INVALID),
    (dict(status=0x70002), ALIGN),
])
def test_refusals_of_write(lib, kw, expect):
    assert write(lib, **kw) == expect


def test_no_rows_is_fine(lib):
    assert write(lib, n=0, slots=None, rows=None) == 0
    assert read(lib, n=0, slots=None, rows=None) == 0


def test_binding_refuses_host_tensors(lib):
    c = W.PagedCache(torch.zeros((2, 64 * 528), dtype=torch.uint8), 64, W.FMT_FP8_528)
    with pytest.raises(B.DsaError):
        B.dsa_cache_write(c, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 512))
    with pytest.raises(B.DsaError):
        B.dsa_cache_read(c, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 512))


def test_binding_takes_tensors_and_numbers(lib):
    """Arguments of another kind raise; what is wrong first decides how."""
    c = W.PagedCache(torch.zeros((2, 64 * 528), dtype=torch.uint8), 64, W.FMT_FP8_528)
    for cache in (c, W.PagedCache([1, 2], 64, W.FMT_FP8_528)):
        with pytest.raises((AttributeError, TypeError, B.DsaError)):
            B.dsa_cache_read(cache, [0, 1, 2], torch.zeros(3, 512))
        with pytest.raises((AttributeError, TypeError, B.DsaError)):
            B.dsa_cache_write(cache, torch.zeros(3, dtype=torch.int32), None)
    with pytest.raises(TypeError):
        B.dsa_cache_write(c, torch.zeros(3, dtype=torch.int32), torch.zeros(3, 512), norm_eps="small")


def test_no_rows_with_a_table_is_fine(lib):
    """A step without new keys: empty arrays, whose address may be null."""
    assert write(lib, n=0, slots=None, rows=None, pos=None, table=0x50000, table_rows=4) == 0
    assert write(lib, n=0, slots=None, rows=None, pos=0x40000, table=0x50000, table_rows=4) == 0
