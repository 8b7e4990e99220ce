"""The marshalling extension: which file it is, and who needs it. No GPU."""
import ctypes
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD


def test_extension_carries_the_interpreters_tag():
    """A copy built for another Python has another name and is not loaded."""
    BLD.build()
    assert B.MARSHAL_PATH == BLD.MARSHAL and os.path.exists(BLD.MARSHAL)
    name = os.path.basename(BLD.MARSHAL)
    assert name.startswith("_marshal.cpython-") and name.endswith(importlib.machinery.EXTENSION_SUFFIXES[0])


def test_decode_does_without_the_extension():
    """Loading, planning and the decode calls; a cache call names what it misses."""
    BLD.build()
    code = """
import torch
from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import workloads as W
B.MARSHAL_PATH = B.MARSHAL_PATH + ".missing"
B.load()
B.dsa_decode_plan(4, 16, 128, num_sms=152)
B.dsa_prefix_plan(4, 16, 128, 152)
c = W.PagedCache(torch.zeros((2, 64 * 528), dtype=torch.uint8), 64, W.FMT_FP8_528)
try:
    B.dsa_cache_read(c, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 512))
except RuntimeError as e:
    print("missing" in str(e) and "build" in str(e) and not isinstance(e, B.DsaError))
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=BLD.ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "True", r.stderr


def test_build_without_python_headers(monkeypatch, tmp_path, capsys):
    lib = BLD.build()
    paths = dict(sysconfig.get_paths(), include=str(tmp_path))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    monkeypatch.setattr(BLD, "MARSHAL", str(tmp_path / "_marshal.so"))
    assert BLD.build() == lib
    assert "Python.h" in capsys.readouterr().err and not os.path.exists(BLD.MARSHAL)


class Array:
    """What the extension asks a tensor for, on device 0."""

    def __init__(self, dtype, shape, ptr=0x10000):
        self.dtype, self.shape, self.ptr = dtype, tuple(shape), ptr

    def stride(self):
        n, s = 1, []
        for e in reversed(self.shape):
            s.append(n)
            n *= e
        return tuple(reversed(s))

    def get_device(self):
        return 0

    def data_ptr(self):
        return self.ptr


class Desc(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("format", ctypes.c_int32)]


@pytest.fixture()
def own(tmp_path):
    """A copy of the extension that takes ``Array`` for tensors (dtypes by name)."""
    BLD.build()
    path = shutil.copy(BLD.MARSHAL, tmp_path)
    loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
    loader.exec_module(m)
    m.setup("u8", "i32", "i64", "bf16", "f16", "f32", lambda: 0, lambda device: 7)
    return m


READ = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.POINTER(Desc), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                        ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p)
WRITE = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.POINTER(Desc), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                         ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p)


def test_numbers_are_not_cut_to_32_bits(own):
    """A page size, format or style of 2^32 + x is refused, not taken as x."""
    seen = []

    def read(desc, slots, n, rows, stride, type_, stream):
        seen.append((desc.contents.page_size, desc.contents.format, n, stride, type_, stream))
        return 0

    def write(desc, slots, n, rows, stride, type_, w, eps, pos, cs, table, style, status, stream):
        seen.append((desc.contents.page_size, desc.contents.format, style))
        return 0

    f_read, f_write = READ(read), WRITE(write)
    a_read, a_write = (ctypes.cast(f, ctypes.c_void_p).value for f in (f_read, f_write))
    slots, rows = Array("i32", (4,)), Array("f32", (4, 512))
    data = Array("u8", (2, 64 * 528))

    def call_read(data=data, page=64, fmt=0):
        return own.cache_read(a_read, data, page, fmt, slots, rows, None)

    def call_write(page=64, fmt=0, style=1):
        return own.cache_write(a_write, data, page, fmt, slots, rows, None, 0.0, None, None, style, None, None)

    assert call_read() == 0 and seen.pop() == (64, 0, 4, 512, 2, 7)
    assert call_write() == 0 and seen.pop() == (64, 0, 1)
    narrow = Array("u8", (2, 64))            # narrower than its pages
    for d in (data, narrow):
        for big in (1 << 32, (1 << 32) + 64, -(1 << 32), 1 << 31, 1 << 62, 1 << 70):
            assert call_read(data=d, page=big) == own.BAD_TENSOR
            assert call_read(data=d, fmt=big) == own.BAD_TENSOR
    for big in (1 << 32, (1 << 32) + 1, -(1 << 32), 1 << 70):
        assert call_write(style=big) == own.BAD_TENSOR
        assert call_write(fmt=big) == own.BAD_TENSOR
    assert call_read(data=narrow) == own.BAD_TENSOR and seen == []
    with pytest.raises(TypeError):
        call_read(fmt="fp8")
