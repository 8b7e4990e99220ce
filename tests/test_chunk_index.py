"""Index arithmetic of the chunk kernels (csrc/dsa_chunk_index.cuh), compiled as
plain C++: every row tile's units cover the keys that its rows attend, and lie
in the halves that the gather writes and the plan holds. No GPU."""
import ctypes
import os
import random
import subprocess

import pytest

from swa_paged_decode_gb300 import build as BLD

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("index") / "chunk_index.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", BLD.CSRC, "-o", lib,
                    os.path.join(HERE, "chunk_index_host.cpp")], check=True)
    lib = ctypes.CDLL(lib)
    lib.most_row_tiles.restype = lib.most_halves.restype = ctypes.c_longlong
    lib.most_row_tiles.argtypes = [ctypes.c_longlong] * 3
    lib.most_halves.argtypes = [ctypes.c_longlong]
    return lib


def cases():
    rng = random.Random(3)
    out = [(1, 1, 0, 1), (1, 128, 128, 128), (1, 129, 128, 64), (300, 300, 129, 20), (5, 2, 0, 16), (5, 0, 7, 16), (0, 9, 0, 8),
           (7, 2**29, 0, 128), (7, 2**29, 2**31 - 1, 128), (9, 3, 2**31 - 1, 1), (2**20, 1, 1, 1)]
    for _ in range(300):
        n = rng.randint(0, 400)
        out.append((n, rng.randint(0, 1500), rng.choice([0, 1, 2, 64, 127, 128, 129, 500, 4096]), rng.choice([1, 7, 16, 20, 64, 128, 200])))
    return out


def test_units_cover_what_rows_attend(index):
    half = ctypes.c_int(0)
    for n, length, window, H in cases():
        tiles = index.seq_tiles(n, length, window, H)
        assert tiles == -(-n * H // 128)
        lo, hi = index.gather_begin(n, length, window), index.gather_end(n, length, window)
        if not index.seq_any(n, length, window):
            assert n == 0 or length == 0
        else:
            assert 0 <= lo < hi <= index.most_halves(length)
        for i in range(tiles) if tiles < 2000 else (0, tiles - 1):
            rows = index.tile_rows(n, length, window, H, i)
            assert rows == min(128, n * H - 128 * i)
            units = index.tile_units(n, length, window, H, i, ctypes.byref(half))
            first, last = (length - n + (128 * i + r) // H for r in (0, rows - 1))
            if last < 0:
                assert units == 0
                continue
            begin = max(0, first - window + 1) if window else 0
            assert units >= 1 and half.value == begin // 128
            # the last row's key is in the last unit, and no unit lies past it
            assert 128 * (half.value + 2 * units) > last >= 128 * (half.value + 2 * units - 2)
            assert lo <= half.value and half.value + 2 * units <= hi


@pytest.mark.parametrize("H", [1, 20, 64, 128, 200])
def test_row_tiles_of_any_split_fit_the_plan(index, H):
    rng = random.Random(H)
    for _ in range(200):
        T, B = rng.randint(0, 300), rng.randint(0, 20)
        cuts = sorted(rng.randint(0, T) for _ in range(B + 1))
        tiles = sum(index.seq_tiles(b - a, 10, 0, H) for a, b in zip(cuts, cuts[1:]))
        assert tiles <= index.most_row_tiles(T, H, B)
