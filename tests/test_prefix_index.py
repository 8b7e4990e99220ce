"""Index arithmetic of the shared-prefix kernels (csrc/dsa_prefix_index.cuh),
compiled as plain C++: every load that the merge makes for a row lies in the
plan's workspace, and the pairs' ranges cover every unit once. No GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    BLD.build()
    lib = str(tmp_path_factory.mktemp("index") / "prefix_index.so")
    # a division by zero or an overflow ends the process, on every machine
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", BLD.CSRC, "-o", lib,
                    os.path.join(HERE, "prefix_index_host.cpp")], check=True)
    path, lib = lib, ctypes.CDLL(lib)
    lib.path = path
    lib.part_loaded.restype = lib.part_slot.restype = lib.schedule_begin.restype = ctypes.c_int64
    return lib


PLANS = [(1, 1, 1, 512), (1, 8, 256, 512), (3, 16, 200, 512), (32, 64, 256, 512), (128, 128, 256, 512),
         (13, 20, 256, 576), (13, 20, 1, 576), (4, 64, 8192, 512)]


@pytest.mark.parametrize("T,H,width,d", PLANS)
def test_merge_loads_lie_in_the_workspace(index, T, H, width, d):
    """Rows without parts (an empty prefix: c0 = 0, c1 = -1) and with 1, 2 and
    all of the pairs, both forms of the merge (a group's parts g, g + groups,
    .. with 2 or 8 of them in flight)."""
    plan, nbytes = B.dsa_prefix_plan(T, H, width, 152, d)
    end = (nbytes - plan.ws_part_o_offset) // 2048
    assert end == 256 * plan.pairs
    for c0, c1 in {(0, -1), (0, 0), (0, plan.pairs - 1), (plan.pairs - 1, plan.pairs - 1)}:
        for late in (0, 128):
            for row in (0, 1, 127):
                for groups, flight in ((1, 2), (2, 8)):
                    for i0 in range(0, max(1, c1 - c0 + 1), groups * flight):
                        for g in range(groups):
                            for i in range(flight):
                                s = index.part_loaded(c0, c1, late, row, i0 + g + groups * i)
                                assert 0 <= s < end, (c0, c1, late, row, i0, g, i, s)


def test_parts_are_the_pairs_slots(index):
    for i in range(5):                        # pair 3 began before the tile, 4 .. 7 with it
        assert index.part_slot(3, 7, 128, 9, i) == (3 + i) * 256 + 9 + (128 if i == 0 else 0)
        assert index.part_loaded(3, 7, 128, 9, i) == index.part_slot(3, 7, 128, 9, i)
    assert index.part_loaded(3, 7, 128, 9, 11) == index.part_slot(3, 7, 128, 9, 4)


def test_no_units_without_keys(index):
    """In a process of its own: a division by zero would end it."""
    code = ("import ctypes, sys; f = ctypes.CDLL(sys.argv[1]).schedule_begin; f.restype = ctypes.c_int64; "
            "print(sum(abs(f(R, 0, C, c)) for R in (1, 5, 1 << 20) for C in (1, 2, 76) for c in (0, 1, C)))")
    r = subprocess.run([sys.executable, "-c", code, index.path], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "0", (r.returncode, r.stdout, r.stderr)


@pytest.mark.parametrize("R,KT,C", [(1, 1, 1), (1, 2, 2), (5, 5, 14), (4, 32, 76), (16, 16, 76), (128, 64, 76), (3, 7, 20),
                                    (1, 256, 76), (1 << 24, 1, 76), (1 << 10, 1 << 21, 76), (97, 2, 700)])
def test_ranges_cover_every_unit_once(index, R, KT, C):
    b = [index.schedule_begin(R, KT, C, c) for c in range(C + 1)]
    assert b[0] == 0 and b[-1] == R * KT and all(x <= y for x, y in zip(b, b[1:]))
    most = max(y - x for x, y in zip(b, b[1:]))
    assert most <= -(-R * (KT + 2) // C) + 1
