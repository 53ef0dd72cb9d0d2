"""The eviction by accumulated weight against its definition: which tokens are
kept (weights, ties, NaN and infinities, the recent window), their order and
lists, the moved rows bit for bit, and everything that is left alone."""
import math

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, Batch, share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def with_room(bt, max_keep):
    """The batch's pools with pages to move into, and their table."""
    kp = max(1, -(-(-(-max_keep // bt.N)) // bt.page))
    extra = bt.B * kp
    grown = []
    for t in (bt.k_pages, bt.v_pages):
        new = torch.randn((bt.N, bt.num_pages + extra, *t.shape[2:]), device=DEV).to(t.dtype)
        new[:, :bt.num_pages] = t
        grown.append(new)
    table = torch.arange(extra, device=DEV, dtype=torch.int32).flip(0).reshape(1, bt.B, kp) + bt.num_pages
    return grown[0], grown[1], table.repeat(bt.N, 1, 1).contiguous()


def pick(acc, L, keep, recent, r, N):
    """Kept local indices, in order."""
    m, want = share(L, r, N), share(min(L, keep), r, N)
    late = [i for i in range(m) if i * N + r >= L - recent]
    take = late[len(late) - min(want, len(late)):]
    a = [(-x if x == x else math.inf, not x == x) for x in acc[:m].tolist()]
    older = sorted(range(m - len(late)), key=lambda i: (a[i][1], a[i][0], i))
    return sorted(older[: want - len(take)] + take)


def run(bt, acc, keep, recent, max_keep=None, spoil=None):
    max_keep = max(keep) if max_keep is None else max_keep
    kp, vp, dst = with_room(bt, max_keep)
    if spoil:
        spoil(bt, dst)
    kcap = max(1, -(-max_keep // bt.N))
    kept = torch.full((bt.N, bt.B, bt.Hkv, kcap + 2), -9, dtype=torch.int32, device=DEV)
    out = torch.full((bt.N, bt.B, bt.Hkv, kcap + 2), 5.0, device=DEV)
    want_k, want_v, want_kept, want_out = kp.clone(), vp.clone(), kept.clone(), out.clone()
    pages = kp.shape[1]
    for b, (_, L) in enumerate(bt.lens):
        if keep[b] < 0:
            continue
        for r in range(bt.N):
            for h in range(bt.Hkv):
                ids = pick(acc[r, b, h], L, min(keep[b], max_keep), recent, r, bt.N)
                for n, i in enumerate(ids):
                    want_kept[r, b, h, n], want_out[r, b, h, n] = i, acc[r, b, h, i]
                    to, at = int(dst[r, b, n // bt.page]), int(bt.block_table[r, b, i // bt.page])
                    if not 0 <= to < pages:
                        continue
                    inside = 0 <= at < pages
                    want_k[r, to, n % bt.page, h] = kp[r, at, i % bt.page, h] if inside else 0
                    want_v[r, to, n % bt.page, h] = vp[r, at, i % bt.page, h] if inside else 0
    binding.cache_evict_paged(kp, vp, bt.block_table, bt.seq_lens, bt.max_len, acc,
                              torch.tensor(keep, dtype=torch.int32, device=DEV), max_keep, recent, dst, kept, out)
    torch.cuda.synchronize()
    assert torch.equal(kept, want_kept)
    assert torch.equal(out.view(torch.int32), want_out.view(torch.int32))
    assert torch.equal(kp.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(vp.view(torch.int16), want_v.view(torch.int16))


def random_acc(bt, levels=None):
    acc = torch.empty((bt.N, bt.B, bt.Hkv, bt.cap), device=DEV).exponential_(1.0)
    return (acc * levels).round() / levels if levels else acc


CASES = [
    # lens, N, Hkv, D, page, keep, recent
    ([(0, 1)], 1, 1, 64, 1, [1], 0),
    ([(0, 40), (0, 7), (0, 0), (0, 33)], 3, 2, 128, 8, [17, 7, 4, 0], 5),
    ([(0, 300), (0, 513)], 2, 2, 128, 16, [100, -1], 64),
    ([(0, 700)], 1, 3, 128, 64, [512], 0),
    ([(0, 1100), (0, 64)], 2, 1, 256, 4, [40, 64], 300),     # the window holds more than is kept
    ([(0, 90)], 4, 2, 64, 2, [90], 10),                       # everything stays
    ([(0, 90)], 4, 2, 64, 2, [5000], 1000),
    ([(0, 2100), (0, 1025)], 1, 2, 72, 32, [1024, 1000], 1),
]


@pytest.mark.parametrize("lens,N,Hkv,D,page,keep,recent", CASES)
@pytest.mark.parametrize("levels", [None, 2])
def test_kept_tokens_and_moved_rows(lens, N, Hkv, D, page, keep, recent, levels):
    bt = Batch(lens, N, Hkv, Hkv, D, page, torch.bfloat16, 0, seed=len(lens) + D)
    run(bt, random_acc(bt, levels), keep, recent)


def test_equal_weights_keep_the_first_tokens():
    bt = Batch([(0, 1200)], 1, 1, 1, 64, 16, torch.float16, 0, seed=31)
    run(bt, torch.zeros((1, 1, 1, 1200), device=DEV), [500], 0)
    acc = torch.zeros((1, 1, 1, 1200), device=DEV)
    acc[..., ::3] = -0.0         # the same value
    run(bt, acc, [500], 20)


def test_nan_is_evicted_first_and_infinities_are_values():
    bt = Batch([(0, 600), (0, 100)], 2, 2, 2, 64, 16, torch.float16, 0, seed=32)
    acc = random_acc(bt, 4)
    acc[:, :, :, 3::7] = math.nan
    acc[:, :, :, 5::11] = math.inf
    acc[:, :, :, 6::13] = -math.inf
    acc[:, :, :, 20:30] *= -1
    run(bt, acc, [200, 20], 16)
    run(bt, acc, [590, 98], 4)
    run(bt, torch.full_like(acc, math.nan), [100, 10], 4)


def test_max_keep_bounds_what_is_kept():
    bt = Batch([(0, 200), (0, 30)], 2, 2, 2, 64, 16, torch.float16, 0, seed=33)
    run(bt, random_acc(bt), [150, 30], 8, max_keep=64)


def test_bad_pages_are_neither_read_nor_written():
    bt = Batch([(0, 200), (0, 90)], 2, 2, 2, 64, 8, torch.float16, 0, seed=34)

    def spoil(bt, dst):
        dst[0, 0, 1], dst[1, 1, 0] = -1, 2 ** 31 - 1
        bt.block_table[0, 1, 2], bt.block_table[1, 0, 0] = 2 ** 31 - 1, -5

    run(bt, random_acc(bt), [100, 60], 16, spoil=spoil)


def test_long_requests():
    bt = Batch([(0, 30011)], 1, 2, 2, 64, 64, torch.bfloat16, 0, seed=35)
    run(bt, random_acc(bt), [9000], 500)
    run(bt, random_acc(bt, 1), [4097], 0)
    # few distinct leading bits: the selection has to go to the last pass
    acc = 1.0 + torch.randint(0, 64, (1, 1, 2, bt.cap), device=DEV).float() * 2.0 ** -23
    run(bt, acc, [12345], 100)


def test_graph_replay_follows_weights_and_lengths():
    bt = Batch([(0, 300)], 2, 2, 2, 64, 16, torch.float16, 0, seed=36)
    acc = random_acc(bt)
    kp, vp, dst = with_room(bt, 100)
    keep = torch.tensor([100], dtype=torch.int32, device=DEV)
    kept = torch.full((2, 1, 2, 50), -9, dtype=torch.int32, device=DEV)
    out = torch.zeros((2, 1, 2, 50), device=DEV)
    args = (kp, vp, bt.block_table, bt.seq_lens, bt.max_len, acc, keep, 100, 10, dst, kept, out)
    binding.cache_evict_paged(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.cache_evict_paged(*args)
    acc.copy_(random_acc(bt))
    keep.fill_(61)
    bt.seq_lens.fill_(211)
    kept.fill_(-9)
    graph.replay()
    torch.cuda.synchronize()
    for r in range(2):
        for h in range(2):
            ids = pick(acc[r, 0, h], 211, 61, 10, r, 2)
            assert kept[r, 0, h].tolist() == ids + [-9] * (50 - len(ids))
