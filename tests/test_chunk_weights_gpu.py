"""The accumulated attention weights against their definition in 64 bits: ragged
batches, tile edges, new tokens that start from zero, rows without a finite
log-sum-exp, NaN keys, entries that are left alone, graphs."""
import math

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, Batch, assert_within, share, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def merged_lse(bt):
    """[T, H] fp32: log-sum-exp of every new token over all ranks' visible tokens."""
    out = torch.zeros((bt.T, bt.H), dtype=torch.float64, device=DEV)
    for b, (n, l) in enumerate(bt.lens):
        for h in range(bt.H):
            parts = []
            for r in range(bt.N):
                s, _ = bt.scores(b, r, h)
                seen = torch.arange(s.shape[1], device=DEV)[None] < bt.limits(b, r)[:, None]
                parts.append(torch.where(seen, s, torch.full_like(s, -math.inf)))
            if n:
                out[bt.rows(b), h] = torch.logsumexp(torch.cat(parts, 1), 1)
    return out.float()


def call(bt, lse, acc, **kw):
    binding.attention_weights_paged(bt.q, bt.k_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len, lse,
                                    acc, bt.scale, **kw)


def start(bt, extra=0):
    acc = torch.rand((bt.N, bt.B, bt.Hkv, bt.cap + extra), device=DEV) * 3
    for b, (n, l) in enumerate(bt.lens):     # what stands where the new tokens go does not matter
        for r in range(bt.N):
            acc[r, b, :, share(l - n, r, bt.N):share(l, r, bt.N)] = math.nan
    return acc


def run(bt, lse, base="e", extra=0):
    acc = start(bt, extra)
    want, tol = weights(bt, lse, acc)
    call(bt, lse / math.log(2.0) if base == "2" else lse, acc, base=base)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    if base == "2":       # the division above rounds: 2^-24 of the log-sum-exp
        tol = tol + want.nan_to_num(0.0).abs() * 2.0 ** -23 * lse.nan_to_num(0.0, 0.0, 0.0).abs().max().item()
    assert_within(acc, want, tol, "acc")
    return acc


BF, HF = torch.bfloat16, torch.float16
CASES = [
    ([(1, 1)], 1, 1, 1, 64, 1, BF, 0, False),
    ([(1, 1), (1, 2), (1, 3), (0, 5), (2, 2)], 4, 4, 2, 128, 8, BF, 3, False),
    ([(1, 63), (1, 64), (1, 65), (1, 127), (1, 129), (1, 257), (1, 700)], 1, 8, 1, 128, 16, HF, 0, False),
    ([(17, 300), (0, 40), (130, 131), (5, 5)], 3, 16, 2, 128, 32, BF, 1, True),
    ([(33, 700), (1, 2000)], 8, 16, 1, 128, 64, HF, 0, False),
    ([(40, 90), (3, 500)], 2, 12, 1, 128, 8, BF, 0, False),
    ([(9, 200), (70, 77)], 2, 6, 2, 64, 16, BF, 2, True),
    ([(300, 460), (1, 30)], 2, 8, 8, 64, 128, HF, 0, False),
    ([(50, 120), (2, 301)], 2, 4, 2, 256, 16, BF, 1, True),
    ([(20, 50)], 5, 6, 1, 256, 4, HF, 0, False),
    ([(30, 65), (1, 9)], 3, 8, 2, 128, 2, BF, 0, True),
    ([(11, 100)], 2, 64, 1, 128, 16, BF, 0, False),
    ([(11, 100)], 2, 48, 1, 128, 16, BF, 0, False),
    ([(600, 1400)], 1, 4, 2, 128, 64, BF, 0, False),
]


@pytest.mark.parametrize("lens,N,H,Hkv,D,page,dtype,pad,strided", CASES)
def test_weights_match_the_definition(lens, N, H, Hkv, D, page, dtype, pad, strided):
    bt = Batch(lens, N, H, Hkv, D, page, dtype, pad, seed=N + H + D, strided=strided, qscale=1.5)
    lse = merged_lse(bt)
    acc = run(bt, lse, "2" if pad else "e", extra=5 if pad else 0)
    # every row of queries gives 1 in all, so the new weights of a request sum to its rows
    if len(lens) == 1 and lens[0][0] == lens[0][1]:
        assert abs(acc.sum().item() - lens[0][0] * H) < 1e-3 * H


@pytest.mark.parametrize("D,page", [(128, 16), (64, 8), (256, 8)])
def test_more_requests_and_ranks_than_threads_of_a_block(D, page):
    lens = [(b % 4, 3 + b % 4 + 13 * b % 97) for b in range(450)]
    lens[200] = (33, 6000)
    bt = Batch(lens, 3, 4, 2, D, page, BF, 1, seed=D)
    run(bt, merged_lse(bt))


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (256, 16)])
def test_rows_without_a_finite_log_sum_exp_add_nothing(D, page):
    bt = Batch([(9, 400), (200, 260)], 2, 8, 2, D, page, BF, 0, seed=21)
    lse = merged_lse(bt)
    lse[2, 3], lse[5, 0], lse[7] = math.nan, -math.inf, math.inf
    lse[100:110] = math.nan
    bt.q[7] = math.nan          # as the row's own NaN leaves it
    bt.q[100, 1] = math.inf
    want_nan = bt.q.isfinite().all(-1)
    q0 = bt.q.clone()
    acc = start(bt)
    bt.q = torch.where(want_nan[..., None], bt.q, torch.zeros_like(bt.q))
    want, tol = weights(bt, lse, acc)
    bt.q = q0
    call(bt, lse, acc)
    torch.cuda.synchronize()
    assert_within(acc, want, tol, "acc")


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (256, 16)])
def test_a_nan_key_spoils_its_own_weight_only(D, page):
    bt = Batch([(9, 400), (150, 260)], 2, 8, 2, D, page, BF, 0, seed=22)
    lse = merged_lse(bt)
    bt.k[0][100, 1, 3] = math.nan
    bt.k[1][255, 0, 0] = math.nan
    bt.fill()
    acc = start(bt)
    want, tol = weights(bt, lse, acc)
    call(bt, lse, acc)
    torch.cuda.synchronize()
    want[0, 0, 1, 50], want[1, 1, 0, 127] = math.nan, math.nan
    assert_within(acc, want, torch.nan_to_num(tol, nan=0.0), "acc")


def test_calls_accumulate_and_repeat_bit_for_bit():
    bt = Batch([(3, 700), (90, 300)], 2, 8, 2, 128, 16, BF, 0, seed=23)
    lse = merged_lse(bt)
    a, b = (torch.zeros((2, 2, 2, bt.cap), device=DEV) for _ in range(2))
    call(bt, lse, a)
    call(bt, lse, b)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    call(bt, lse, a)
    torch.cuda.synchronize()
    for i, (n, l) in enumerate(bt.lens):
        for r in range(2):
            m, old = share(l, r, 2), share(l - n, r, 2)
            assert torch.allclose(a[r, i, :, :old], 2 * b[r, i, :, :old], rtol=2e-7, atol=0)
            assert torch.equal(a[r, i, :, old:m], b[r, i, :, old:m])
            assert bool((a[r, i, :, m:] == 0).all())


def test_graph_replay_and_bad_pages():
    bt = Batch([(3, 700), (90, 300)], 2, 8, 2, 128, 16, BF, 2, seed=24)
    lse = merged_lse(bt)
    bt.block_table[1, 0, 3] = -7
    i = torch.arange(48, 64, device=DEV)
    bt.k[0][i * 2 + 1] = 0
    acc = start(bt)
    acc0 = acc.clone()
    call(bt, lse, torch.zeros_like(acc))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(bt, lse, acc)
    acc.copy_(acc0)
    graph.replay()
    torch.cuda.synchronize()
    want, tol = weights(bt, lse, acc0)
    assert_within(acc, want, tol, "acc")
