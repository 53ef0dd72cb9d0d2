"""The bits of a request's chunk attention do not depend on what else lies in the query tensor or in shared memory:
the rows of the next request, the padding behind the batch, and rows of a block that no query fills."""
import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def call(bt, q):
    o = torch.full((bt.N, bt.T, bt.H, bt.D), 7.0, dtype=bt.dtype, device=DEV)
    lse = torch.full((bt.N, bt.T, bt.H), 7.0, device=DEV)
    binding.extend_attention_paged(q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len,
                                   o, lse, bt.scale)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    return o, lse


@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (256, 16)])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (12, 1), (16, 2)])
def test_rows_of_other_requests_and_padding_leave_the_bits(H, Hkv, D, page):
    # single tokens and drafts between rows whose scores are beyond 2^16 (or infinite, or not a number) in one call
    # and ordinary in the other
    lens = [(1, 700), (3, 900), (1, 1200), (9, 400), (2, 333)]
    bt = Batch(lens, 2, H, Hkv, D, page, torch.bfloat16, pad=7, seed=H + D)
    want = call(bt, bt.q)
    for mine in range(len(lens)):
        for value in (1e7, -3e6, float("inf"), float("nan")):
            q = torch.full_like(bt.q, value)
            q[bt.rows(mine)] = bt.q[bt.rows(mine)]
            got = call(bt, q)
            assert torch.equal(got[0][:, bt.rows(mine)], want[0][:, bt.rows(mine)])
            assert torch.equal(got[1][:, bt.rows(mine)], want[1][:, bt.rows(mine)])


@pytest.mark.parametrize("H", [12, 48, 5])
@pytest.mark.parametrize("D", [128, 64])
def test_equal_calls_where_a_block_has_rows_that_no_query_fills(H, D):
    # 128 is no multiple of the group: the last rows of a block keep what the shared memory held before, here the
    # rows of another call whose scores are huge
    bt = Batch([(1, 3000), (40, 900), (2, 50)], 2, H, 1, D, 16, torch.bfloat16, seed=H)
    other = Batch([(300, 900)], 1, 4, 1, D, 16, torch.bfloat16, seed=1)
    want = call(bt, bt.q)
    for scale in (1.0, 1e7, -1e7):
        call(other, (other.q.float() * scale).to(torch.bfloat16))
        got = call(bt, bt.q)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
