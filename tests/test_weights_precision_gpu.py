"""Single attention weights against the bound that the header states: off by a
factor e^d, |d| <= 2^-16 A + 2^-22 (1 + |s| + |lse|), A the sum of the product's
magnitudes, at scores from near zero to far beyond what a softmax holds. The
bound: the tensor core adds at most 576 exact products in 36 steps, each off by
2^-22 of A, and the sums of the blocks add 2^-22 of it; score and lse are each
rounded twice on their way to base 2 and once together (4 times 2^-24 of them),
the exponential is good to 2^-22. Query elements below 2^-14 of their row's largest
add 2^-25 of it times the key. One head and one token to a list: an entry's score
is one weight; what lies below fp32's normal range may be zero."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from swa_paged_decode_gb300 import workloads as W
from tests._serve_ref import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("fmt", list(W.RECORD_BYTES))
@pytest.mark.parametrize("q_log2", [-6, 0, 3, 5])
@pytest.mark.parametrize("shift", [0.0, 40.0])
@pytest.mark.parametrize("sink", [False, True])
def test_single_weights(fmt, q_log2, shift, sink):
    c = Batch([(1, 700), (1, 129), (1, 1000)], 1, fmt, seed=fmt + 7, q_log2=q_log2, sink=sink)
    rows = [x for x in c.scores()]
    lse = torch.stack([torch.logsumexp(x[4][0, 0], 0) for x in rows]).float()[:, None] + shift
    out = torch.zeros((c.B, c.width), device="cuda")
    attn = B.AttentionWeights(c.T, c.B, 1, c.width, "cuda", c.d)
    attn(c.q, c.cache, c.slots, c.lengths, c.starts, lse, None, out, c.scale, 0, c.sink)
    torch.cuda.synchronize()
    assert B.dsa_decode_read_status(attn.workspace) == 0
    for b, t, at, k, x, mass in rows:
        s, l, q = x[0, 0], lse[b, 0].double(), c.queries()[t, 0]
        den = l if c.sink is None else torch.logaddexp(l, c.sink[0].double())
        small = c.scale * q.abs().max() * k.abs().sum(1) * 2.0 ** -25
        d = 2.0 ** -16 * mass[0, 0] + 2.0 ** -22 * (1 + s.abs() + den.abs()) + small
        want = (s - den).exp()
        tol = want * torch.expm1(d) + 2.0 ** -126
        err = (out[b, at].double() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
