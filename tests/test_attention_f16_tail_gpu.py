"""fp16 chunk attention of a row with one dominant token and a long flat tail far below it: the tail's weights are
below what an fp16 holds beside 1, and their sum is not."""
import math

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, Batch, assert_within, attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


@pytest.mark.parametrize("below", [10.0, 14.0, 17.4, 18.0])
@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (128, 4), (256, 32)])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("n", [1, 40])
def test_a_long_tail_keeps_its_mass(below, D, page, far, n):
    tail = 30000
    H = 2 if n == 1 else 4      # one row block of two tiles at a time, or pairs of blocks
    bt = Batch([(n, tail)], 1, H, 1, D, page, torch.float16, seed=5)
    bt.scale = 1.0
    # the scores: `below` for the first token, 0 for the tail; with `far` both moved by 2^17 (exact in 32 bits: the
    # fp16 of `below` is a multiple of 2^-6)
    bt.q.zero_()
    bt.q[..., 0] = 1.0
    bt.q[..., 1] = 256.0 if far else 0.0
    bt.k[0].zero_()
    bt.k[0][0, :, 0] = below
    bt.k[0][:, :, 1] = 512.0
    bt.v[0].fill_(100.0)
    bt.v[0][:, :, 1::2] = -37.0
    bt.v[0][0] = 0.0
    bt.fill()
    o = torch.empty((1, bt.T, H, D), dtype=torch.float16, device=DEV)
    lse = torch.empty((1, bt.T, H), device=DEV)
    binding.extend_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens,
                                   bt.max_len, o, lse, bt.scale)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    want, want_lse, o_tol, lse_tol = attention(bt)
    # (with `far` the bounds of a 32-bit score at 2^17 hold: the log-sum-exps by which parts are joined are rounded
    # to 2^-7 powers of two there)
    # a weight below fp16's normal range is off by half its step of 2^-24, beside 2^7 for the row's largest (2^15 in
    # the register-tiled kernel); the row's sum is at least that largest one
    tc = D < 256 and page >= 8
    o_tol = o_tol + 2.0 ** (-32 if tc else -40) * bt.v[0].double().abs().sum(0).amax()
    assert_within(o, want, o_tol, "o")
    assert_within(lse, want_lse, lse_tol, "lse")


@pytest.mark.parametrize("D,page", [(128, 16), (64, 16), (128, 4), (256, 16)])
@pytest.mark.parametrize("step", [2.0 ** 20, 2.0 ** 26, 2.0 ** 27, 2.0 ** 28, 2.0 ** 30])
@pytest.mark.parametrize("n", [1, 40])
def test_scores_beyond_what_32_bits_resolve(D, page, step, n):
    """Scores around `step` differ by a few of their own units in the last place, which are many powers of two of
    weight each: whatever they round to, a row's output is a mean of the values it sees."""
    L = 1500
    bt = Batch([(n, L)], 1, 2, 1, D, page, torch.float16, seed=7)
    bt.scale = 1.0
    # 2^a times (2^b + i 2^(b - 10)): rising by an fp16 step of the keys from tile to tile; the queries' second
    # element adds less than that
    a, b = (15, round(math.log2(step)) - 15) if step > 2.0 ** 24 else (10, round(math.log2(step)) - 10)
    i = torch.arange(L, device=DEV)
    bt.q.zero_()
    bt.q[..., 0] = 2.0 ** a
    bt.q[..., 1] = 2.0 ** (a - 11)
    bt.k[0].zero_()
    bt.k[0][:, 0, 0] = (2.0 ** b + (i // 300) * 2.0 ** (b - 10)).to(torch.float16)
    bt.k[0][:, 0, 1] = ((i // 100) % 3 * 2.0 ** (b - 9)).to(torch.float16)
    bt.v[0] = (1 + torch.rand(bt.v[0].shape, generator=bt.g, device=DEV)).to(torch.float16)
    bt.fill()
    for sign in (1.0, -1.0):
        bt.q[..., :2] = bt.q[..., :2].abs() * sign
        o = torch.empty((1, bt.T, 2, D), dtype=torch.float16, device=DEV)
        lse = torch.empty((1, bt.T, 2), device=DEV)
        binding.extend_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens,
                                       bt.max_len, o, lse, bt.scale)
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        assert bool(lse.isfinite().all())
        # P and o are rounded to fp16 once each (2^-11), the values lie in [1, 2]
        assert bool((o >= 1 - 2.0 ** -9).all()) and bool((o <= 2 + 2.0 ** -8).all())
