"""dsa_evict of lists with unused and repeated entries: each competes by its score
and comes out as it stands."""
import pytest
import torch

from swa_paged_decode_gb300 import binding as B
from swa_paged_decode_gb300 import build as BLD
from tests.test_evict_gpu import Lists

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    BLD.build()
    B.load()


@pytest.mark.parametrize("width,budget", [(40, 7), (3000, 1000)])
@pytest.mark.parametrize("what", [-1, 2**31 - 1, 5])
def test_unused_and_repeated_entries(width, budget, what):
    c = Lists([width, width // 2, budget], width, budget, first=2, last=3, seed=width)
    c.slots[torch.rand(c.slots.shape, generator=torch.Generator().manual_seed(1)).cuda() < 0.4] = what
    c.call()
    c.check()
    assert bool((c.freed == what).any()) and bool((c.kept == what).any())
