"""Groups whose first request has ended, or holds less than the others have in common: it asks for nothing, and its
table entries, which name no pages, are not read for the others."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build
from test_prefix_attention_gpu import Shared

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("idle", [[(0, 0)], [(0, 100)], [(0, 0), (0, 0), (0, 2700)]])
def test_the_first_request_holds_less(idle, D, causal):
    n, k = 2770, len(idle)
    bt = Shared(idle + [(1 + b % 2, n + 10 + 3 * b) for b in range(20)], [(k, k + 20, n)], D=D)
    assert bt.block_table[:, 0, -1].ge(bt.num_pages).all()      # no page of the pool
    bt.group_start[0] = 0
    o, lse = bt.run(causal=causal)
    bt.check(o, lse, causal=causal)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_first_request_holds_it_all(D):
    """Then its entries serve, as they did: members' tables name no pages for the common part."""
    n = 2752
    bt = Shared([(0, n)] + [(1, n + 10 + 3 * b) for b in range(20)], [(0, 21, n)], own_entries="bad", D=D)
    bt.check(*bt.run())
