"""Accumulated weights of items that take two and more query tiles, most of whose blocks hold no second tile of
tokens: the two groups of warps that share a tile's sum meet at every item, those of an empty tile at none."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import Batch, assert_within, weights
from test_chunk_weights_gpu import merged_lse, start

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("q,lens", [
    (20, [100] * 400),                                     # two query tiles of 16 new tokens, one tile of tokens
    (20, [100, 200, 90, 120, 256, 40, 300, 128, 129] * 40),
    (40, [60, 100, 250, 128, 130] * 60),                   # three query tiles
    (17, [30, 300, 20, 500, 100, 100] * 40),
])
def test_items_of_several_query_tiles(q, lens, D):
    bt = Batch([(min(q, n), n) for n in lens], 1, 8, 1, D, 16, torch.bfloat16, seed=q + D)
    lse = merged_lse(bt)
    first = start(bt)
    want, tol = weights(bt, lse, first)
    runs = []
    for _ in range(4):
        acc = first.clone()
        binding.attention_weights_paged(bt.q, bt.k_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len, lse,
                                        acc, bt.scale)
        runs.append(acc)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert_within(runs[0], want, tol, "acc")
    for acc in runs[1:]:
        assert torch.equal(acc, runs[0])
