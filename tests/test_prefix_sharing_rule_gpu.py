"""A common part is taken out only where that saves blocks of rows, counted as the kernel that runs cuts them: 64 rows in
the register-tiled kernel (pages under 8 tokens, scales that are not positive), whole tokens of a group's heads.
Members' tables name no pages for the common part here, so the log-sum-exps tell whose entries were read."""
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


# new tokens of a request, common tokens, scale's sign, arguments: every request fills its blocks of rows by itself
ALONE = {
    "pages of four, 64 rows": (8, 1600, 1, dict(page=4, H=8, Hkv=1, D=64)),
    "a negative scale, 128 rows": (16, 3200, -1, dict(H=8, Hkv=1, D=128)),
    "no scale, 128 rows": (16, 3200, 0, dict(H=8, Hkv=1, D=64)),
    "48 heads a group, 192 rows of 256": (4, 8000, 1, dict(H=48, Hkv=1, D=64)),
    "wide heads, 64 rows": (8, 1600, 1, dict(H=8, Hkv=1, D=256)),
}


@pytest.mark.parametrize("name", ALONE)
def test_nothing_is_shared_where_it_saves_nothing(name):
    n, common, sign, kw = ALONE[name]
    bt = Shared([(n, common + n + 3 * b) for b in range(20)], [(0, 20, common)], own_entries="bad", N=1, **kw)
    scale = sign * bt.scale
    o, lse = bt.run(scale=scale)
    o1, lse1 = bt.outputs()
    binding.extend_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len,
                                   o1, lse1, scale)
    # both off by at most 2 err + 2^-20 + 2^-22 |lse|, as chunk_ref has it: far below 2^-12 for these scores, and a
    # thousandth of what the first request's keys make of it (tokens of no page have scores of 0)
    assert (lse - lse1).abs().max() <= 2.0 ** -12
    assert (o.float() - o1.float()).abs().max() <= 2.0 ** -6 * o1.float().abs().max()
    if sign:
        bt.own_entries = "first"
        bt.fill()
        assert (bt.run(scale=scale)[1] - lse)[:, bt.start[1]:].abs().max() > 0.1


@pytest.mark.parametrize("kw,sign", [(dict(page=4, D=64), 1), (dict(D=128), -1), (dict(D=256), 1)])
def test_single_tokens_share(kw, sign):
    bt = Shared([(1, 2810 + 2 * b) for b in range(40)], [(0, 40, 2800)], own_entries="bad", N=1, H=8, Hkv=1, **kw)
    bt.scale *= sign
    bt.check(*bt.run())
