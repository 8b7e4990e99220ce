"""The pairs' walks over a chunk call's row tiles (csrc/dsa_chunk_index.cuh),
compiled as plain C++: the tile that a pair looks ahead at is the one that it
takes next, tiles without keys between them or not, and every unit of every tile
is taken once. No GPU."""
import ctypes
import os
import random
import subprocess

import pytest

from swa_paged_decode_gb300 import build as BLD

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    lib = str(tmp_path_factory.mktemp("walk") / "chunk_walk.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-fsanitize=integer-divide-by-zero,signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", BLD.CSRC, "-o", lib,
                    os.path.join(HERE, "chunk_walk_host.cpp")], check=True)
    f = ctypes.CDLL(lib).walk_batch

    def run(sizes, H, window=0, pairs=1):
        B = len(sizes)
        return f(B, (ctypes.c_int * B)(*[n for n, _ in sizes]), (ctypes.c_int * B)(*[l for _, l in sizes]), window, H, pairs)
    return run


@pytest.mark.parametrize("sizes,H,pairs", [
    ([(1, 200), (1, 0), (1, 200)], 64, 1),                      # an idle request between two
    ([(4, 300), (12, 4), (2, 300)], 32, 1),                     # two whole tiles before the list's start
    ([(1, 0), (1, 0), (1, 200), (1, 0), (1, 0), (1, 200), (1, 0)], 64, 1),
    ([(1, 0), (1, 0)], 64, 3), ([(0, 5), (5, 0)], 128, 2), ([], 16, 2),
    ([(1, 100 if b != 80 else 0) for b in range(160)], 64, 76),
])
def test_tiles_without_keys(walk, sizes, H, pairs):
    assert walk(sizes, H, 0, pairs) == 0


@pytest.mark.parametrize("H", [1, 20, 64, 128, 200])
def test_any_batch(walk, H):
    rng = random.Random(H)
    for _ in range(400):
        sizes = []
        for _ in range(rng.randint(1, 40)):
            n = rng.choice([0, 1, 1, 1, rng.randint(2, 60)])
            sizes.append((n, rng.choice([0, 0, n // 2, n, rng.randint(0, 40), rng.randint(1, 3000)])))
        window = rng.choice([0, 0, 1, 100, 128, 129, 700])
        for pairs in (1, rng.randint(1, 20), 76):
            assert walk(sizes, H, window, pairs) == 0, (sizes, window, pairs)
