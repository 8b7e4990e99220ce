"""Shared-prefix attention where many small weights stand beside a large one.

One key's score lies `gap` above those of all others: each of the others has
weight e^-gap, all of them N e^-gap. The weights are f16 numbers times a power
of two of the row: a weight is off by 2^-11 of itself, or by 2^-32 of the row's
largest where that is more. With the scores' own error delta (below) the
output is off by expm1(2 delta) of the weights' magnitudes, plus these, plus
bf16's half step 2^-8."""
import math

import numpy as np
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("N,gap", [(1 << 18, 17.5), (1 << 18, 12.0), (1 << 16, 16.7), (5000, 9.0)])
@pytest.mark.parametrize("where", [0, -1])
@pytest.mark.parametrize("num_sms", [0, 2])
def test_many_small_weights(N, gap, where, num_sms):
    if num_sms and N > 5000:
        num_sms = 16
    scale = 1.0 / 16
    rows = torch.zeros((2, 512))
    rows[0, 0], rows[0, 100] = 8.0, 1.0      # the large one: score gap
    rows[1, 300], rows[1, 400] = 1.0, -2.0   # the others: score 0
    q = torch.zeros((1, 3, 512))
    q[..., 0] = round(gap / 8.0 / scale * 4) / 4
    gap = float(q[0, 0, 0]) * 8.0 * scale
    cache = W.PagedCache(torch.zeros((1, 64 * 528), dtype=torch.uint8, device="cuda"), 64, W.FMT_FP8_528)
    B.dsa_cache_write(cache, torch.arange(2, dtype=torch.int32, device="cuda"), rows.cuda())
    back = torch.empty((2, 512), device="cuda")
    B.dsa_cache_read(cache, torch.arange(2, dtype=torch.int32, device="cuda"), back)
    v = back.double().cpu().numpy()
    slots = torch.ones(N, dtype=torch.int32, device="cuda")
    slots[where] = 0
    attn = B.PrefixAttention(1, 3, N, "cuda", num_sms=num_sms)
    out, lse = attn(q.to(torch.bfloat16).cuda(), cache, slots, torch.tensor([N], dtype=torch.int32, device="cuda"), scale)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == 0
    s = scale * float(q[0, 0, 0]) * v[0, 0]
    rest = (N - 1) * math.exp(-s)
    want = (v[0] + rest * v[1]) / (1 + rest)
    mag = (np.abs(v[0]) + rest * np.abs(v[1])) / (1 + rest)
    delta = (2.0 ** -10 + 2.0 ** -13) * s + 2.0 ** -17
    small = (np.abs(v[0]) + (N - 1) * np.abs(v[1])) * 2.0 ** -32
    tol = math.expm1(2 * delta) * (mag + np.abs(want)) + 2.0 ** -10 * mag + small
    tol = tol + (np.abs(want) + tol) * 2.0 ** -8
    got = out.double().cpu().numpy()[0]
    assert np.all(np.abs(got - want) <= tol), (got[0, [0, 100, 300, 400]], want[[0, 100, 300, 400]], tol[[0, 100, 300, 400]])
    assert np.all(np.abs(lse.double().cpu().numpy() - (s + math.log1p(rest))) <= delta + 2.0 ** -18 * s)
