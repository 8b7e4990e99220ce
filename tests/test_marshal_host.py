"""The marshalling extension: which file it is, and who needs it. No GPU."""
import importlib.machinery
import os
import subprocess
import sys
import sysconfig

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
