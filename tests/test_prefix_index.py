"""Index arithmetic of the shared-prefix kernels (csrc/dsa_prefix_index.cuh),
compiled as plain C++: every load that the merge makes for a row lies in the
plan's workspace. No GPU."""
import ctypes
import os
import subprocess

import pytest

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    BLD.build()
    lib = str(tmp_path_factory.mktemp("index") / "prefix_index.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I", BLD.CSRC, "-o", lib,
                    os.path.join(HERE, "prefix_index_host.cpp")], check=True)
    lib = ctypes.CDLL(lib)
    lib.part_loaded.restype = lib.part_slot.restype = ctypes.c_int64
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
