"""Shared-prefix attention of several whole row tiles to a CTA pair, the last one
with rows that end inside a warp, with and without a tail."""
import pytest

from swa_paged_decode_gb300 import workloads as W
from tests.test_prefix_gpu import Case, _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,H", [(13, 21), (20, 17), (30, 25)])
def test_whole_tiles(fmt, tail, T, H):
    c = Case(T, H, 400, fmt, seed=T, sink=True, tail=tail, rope=None if fmt == W.FMT_V32_656 else W.ROPE_NEOX)
    for sms in (2, 4):
        out, lse, _ = c.run(num_sms=sms)
        c.check(out, lse)
