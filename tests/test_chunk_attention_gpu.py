"""The attention of a chunk of new tokens over paged round-robin caches against
its definition in 64 bits: ragged batches from empty requests to long ones,
tile edges, every head layout, page sizes and strides, both rules of
visibility, splits, what masked places hold, bad pages, streams and graphs."""
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


def outputs(bt):
    o = torch.full((bt.N, bt.T, bt.H, bt.D), 7.0, dtype=bt.dtype, device=DEV)
    lse = torch.full((bt.N, bt.T, bt.H), 7.0, device=DEV)
    return o, lse


def call(bt, o, lse, **kw):
    binding.extend_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens,
                                   bt.max_len, o, lse, bt.scale, **kw)


def check(bt, o, lse, causal=True, base="e"):
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    want_o, want_lse, o_tol, lse_tol = attention(bt, causal)
    n = bt.start[-1]
    assert bool((o[:, n:] == 7.0).all()) and bool((lse[:, n:] == 7.0).all()), "padding rows written"
    got = lse.double() * (math.log(2.0) if base == "2" else 1.0)
    assert_within(got[:, :n], want_lse[:, :n], lse_tol[:, :n], "lse")
    assert_within(o[:, :n], want_o[:, :n], o_tol[:, :n], "o")


def run(bt, causal=True, base="e"):
    o, lse = outputs(bt)
    call(bt, o, lse, causal=causal, base=base)
    check(bt, o, lse, causal, base)
    return o, lse


BF, HF = torch.bfloat16, torch.float16
CASES = [
    # lens, N, H, Hkv, D, page, dtype, pad, strided
    ([(1, 1)], 1, 1, 1, 64, 1, BF, 0, False),
    ([(1, 1), (1, 2), (1, 3), (0, 5), (2, 2)], 4, 4, 2, 128, 8, BF, 3, False),
    ([(1, 63), (1, 64), (1, 65), (1, 127), (1, 128), (1, 129), (1, 257)], 1, 8, 1, 128, 16, HF, 0, False),
    ([(63, 63), (64, 64), (65, 65), (129, 129)], 1, 4, 4, 128, 16, BF, 0, False),
    ([(17, 300), (0, 40), (130, 131), (5, 5)], 3, 16, 2, 128, 32, BF, 1, True),
    ([(33, 700)], 8, 16, 1, 128, 64, HF, 0, False),
    ([(40, 90), (3, 500)], 2, 12, 1, 128, 8, BF, 0, False),
    ([(9, 200), (70, 77)], 2, 6, 2, 64, 16, BF, 2, True),
    ([(100, 260), (1, 30)], 2, 8, 8, 64, 128, HF, 0, False),
    ([(50, 120), (2, 301)], 2, 4, 2, 256, 16, BF, 1, True),
    ([(20, 50)], 5, 6, 1, 256, 4, HF, 0, False),
    ([(30, 65), (1, 9)], 3, 8, 2, 128, 2, BF, 0, True),
    ([(11, 100)], 2, 64, 1, 128, 16, BF, 0, False),
    ([(11, 100)], 2, 48, 1, 128, 16, BF, 0, False),
    ([(260, 600)], 1, 5, 5, 128, 256, HF, 0, False),
]


@pytest.mark.parametrize("lens,N,H,Hkv,D,page,dtype,pad,strided", CASES)
@pytest.mark.parametrize("causal", [True, False])
def test_partials_match_the_definition(lens, N, H, Hkv, D, page, dtype, pad, strided, causal):
    bt = Batch(lens, N, H, Hkv, D, page, dtype, pad, seed=N + H + D, strided=strided, qscale=1.5)
    run(bt, causal, "2" if pad else "e")


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (256, 32), (128, 4)])
def test_long_requests_are_split_and_joined(D, page):
    # one request of few rows over a long cache: every CTA takes a part of it
    bt = Batch([(2, 40001)], 2, 8, 2, D, page, BF, 0, seed=D, qscale=2.0)
    run(bt)
    # a mix of long and short ones
    bt = Batch([(1, 9000), (70, 5000), (1, 3), (0, 77), (300, 3500), (1, 12000)], 2, 8, 1, D, page, HF, 1, seed=D + 1)
    run(bt)
    bt = Batch([(600, 2000)], 1, 4, 4, D, page, BF, 0, seed=D + 2)
    run(bt, causal=False, base="2")


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (256, 32)])
def test_full_and_partial_row_blocks_share_the_ranges(D, page):
    # every request ends in a block of a few new tokens: their tiles weigh less in the split
    run(Batch([(276, 1500 + 37 * b) for b in range(10)], 2, 4, 4, D, page, HF, 2, seed=D))
    run(Batch([(40, 900 + 100 * b) for b in range(6)], 2, 16, 2, D, page, BF, 0, seed=D + 1), causal=False)


@pytest.mark.parametrize("D,page", [(128, 16), (64, 8), (256, 8)])
def test_more_requests_and_ranks_than_threads_of_a_block(D, page):
    lens = [(b % 4, 3 + b % 4 + 13 * b % 97) for b in range(450)]
    lens[200] = (33, 6000)
    run(Batch(lens, 3, 4, 2, D, page, BF, 1, seed=D))


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (256, 32), (128, 1)])
def test_scores_that_keep_rising(D, page):
    # keys ordered so that the running maximum moves with every tile, by up to hundreds of powers of two
    bt = Batch([(3, 1500), (130, 900)], 1, 4, 1, D, page, BF, 0, seed=9, qscale=0.0)
    bt.q += 1.0
    for b, (_, l) in enumerate(bt.lens):
        up = torch.linspace(-10, 10, l, device=DEV)[:, None, None]
        bt.k[b] = (0.3 * torch.randn(bt.k[b].shape, generator=bt.g, device=DEV) + up).to(BF)
    bt.fill()
    run(bt)


@pytest.mark.parametrize("D,page", [(128, 64), (64, 16), (256, 32), (128, 2)])
@pytest.mark.parametrize("N", [1, 3])
def test_masked_places_may_hold_anything(D, page, N):
    """A token with NaN or infinite K and V reaches the rows that see it, and no others."""
    lens = [(40, 40), (70, 200), (1, 90), (200, 330)]
    bt = Batch(lens, N, 4, 2, D, page, BF, 0, seed=11 + N)
    bt.v[0][25, 0, 3] = math.inf          # rows 25.. see it
    bt.v[0][39, 1, 5] = math.nan          # the last row alone
    bt.v[1][199] = math.nan
    bt.v[3][300, :, 1::2] = -math.inf
    bt.v[3][310, 0, 1] = math.inf
    bt.fill()
    run(bt)
    run(bt, causal=False)
    bt.k[0][30, 0, 2] = math.nan          # a NaN score: the rows that see it are NaN whole
    bt.k[1][198, 1, 0] = math.inf
    bt.fill()
    o, lse = outputs(bt)
    call(bt, o, lse)
    torch.cuda.synchronize()
    r = 30 % N
    rows = o[r, bt.rows(0), 0:2].float()
    assert bool(rows[30:].isnan().all()) and bool(rows[:25].isfinite().all())
    assert bool(lse[r, bt.rows(0), 0:2][30:].isnan().all()) and bool(lse[r, bt.rows(0), 2:].isfinite()[1 * N:].all())


def test_rows_of_scores_at_the_types_lowest_value():
    # every score far below zero: exp(s - lse) is still a softmax
    for D, page in ((128, 16), (64, 8), (256, 16)):
        bt = Batch([(5, 300)], 2, 4, 2, D, page, BF, 0, seed=13)
        bt.q.fill_(1.0)
        for b in range(bt.B):
            bt.k[b].fill_(-2e38 / D)
        bt.fill()
        bt.scale = 1.0
        o, lse = outputs(bt)
        call(bt, o, lse)
        torch.cuda.synchronize()
        assert bool(o.isfinite().all()) and bool(lse.isfinite().all())


@pytest.mark.parametrize("D,page", [(128, 16), (64, 64), (256, 16), (128, 1)])
def test_page_indices_outside_the_pool_read_zero_rows(D, page):
    bt = Batch([(30, 200)], 2, 4, 2, D, page, BF, 0, seed=14)
    for r, j in ((0, 1), (1, 0)):
        bt.block_table[r, 0, j] = bt.num_pages + 5 if r else -1
        i = torch.arange(j * page, min((j + 1) * page, 100), device=DEV)
        bt.k[0][i * 2 + r] = 0
        bt.v[0][i * 2 + r] = 0
    run(bt)


def test_lengths_that_do_not_fit_are_bounded():
    """More new tokens than the length, lengths above the maximum or negative, a query_start that leaves the rows."""
    bt = Batch([(9, 9), (4, 64)], 2, 4, 2, 128, 16, BF, 2, seed=15)
    bt.lens = [(9, 5), (4, 64)]
    bt.seq_lens.copy_(torch.tensor([5, 9000], device=DEV))
    o, lse = run(bt)
    assert bool((lse[:, :4] == -math.inf).all()) and bool((o[:, :4] == 0).all())
    bt.seq_lens.copy_(torch.tensor([-3, 64], device=DEV))
    o, lse = outputs(bt)
    call(bt, o, lse)
    torch.cuda.synchronize()
    assert bool((lse[:, :9] == -math.inf).all()) and bool((o[:, :9] == 0).all())
    bt.query_start.copy_(torch.tensor([0, 9, 1000], device=DEV))
    call(bt, o, lse)
    torch.cuda.synchronize()
    assert binding.device_status() == 0


def test_single_new_tokens_agree_with_the_decode_attention():
    bt = Batch([(1, n) for n in (1, 130, 700, 2000)], 2, 16, 2, 128, 16, BF, 0, seed=16)
    o, lse = run(bt)
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    binding.decode_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.seq_lens, bt.max_len, o2, lse2,
                                   bt.scale, split_tokens=1024)
    torch.cuda.synchronize()
    _, _, o_tol, lse_tol = attention(bt)
    assert bool(((o.double() - o2.double()).abs() <= 2 * o_tol).all())
    assert bool(((lse.double() - lse2.double()).abs().nan_to_num() <= 2 * lse_tol).all())


def test_equal_calls_give_equal_bits_and_streams_do_not_share():
    bt = Batch([(40, 3000), (2, 9000), (300, 700)], 2, 8, 2, 128, 16, BF, 0, seed=17)
    o, lse = run(bt)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [outputs(bt) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (a, b) in zip(streams, outs):
            call(bt, a, b, stream=s)          # its own workspace, not the current stream
            torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(255)   # what the allocator hands out meanwhile
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, o) and torch.equal(b, lse)


def test_graph_replay_follows_the_lengths():
    bt = Batch([(3, 2000), (64, 900), (1, 50)], 2, 8, 2, 128, 16, BF, 4, seed=18)
    o, lse = outputs(bt)
    ws = torch.empty(binding.extend_workspace_bytes(bt.N, bt.B, bt.T, bt.H, bt.Hkv, bt.D, bt.max_len),
                     dtype=torch.uint8, device=DEV)
    call(bt, o, lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(bt, o, lse, workspace=ws)
    ws.fill_(255)
    bt.lens = [(1, 7), (0, 900), (60, 1000)]
    bt2 = Batch(bt.lens, 2, 8, 2, 128, 16, BF, 11, seed=19, max_len=2000)
    for name in ("k_pages", "v_pages", "block_table", "query_start", "seq_lens", "q"):
        src, dst = getattr(bt2, name), getattr(bt, name)
        if name.endswith("pages"):
            dst.fill_(math.nan)
            dst[:, :src.shape[1]] = src
        else:
            dst.copy_(src)
    o.fill_(7.0)
    lse.fill_(7.0)
    graph.replay()
    bt2.T = bt.T
    check(bt2, o, lse)
