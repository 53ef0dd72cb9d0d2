"""Page bookkeeping against its definition in plain integers: every element of
every buffer, what is left alone included."""
import random

import pytest
import torch

import pages_ref as ref
from decode_context_attention_gb300 import binding, build

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device=DEV)


class State:
    """A pool whose tables hold the requests' cached tokens; everything else is a mark."""

    def __init__(self, cached, N, page, max_len, groups=None, seed=0, spare=1 << 20, wide=0, bad=0.0):
        r = random.Random(seed)
        self.N, self.B, self.page, self.max_len, self.groups = N, len(cached), page, max_len, groups
        self.mp = max(1, -(-(-(-max_len // N)) // page)) + wide
        self.cached = cached
        need = [sum(ref.entries(c, k, N, page) for c in cached) for k in range(N)]
        self.num_pages = max(need) + min(spare, 4000) + 5
        self.table = [[[-7] * self.mp for _ in cached] for _ in range(N)]
        self.free, self.count = [], []
        for k in range(N):
            perm = list(range(self.num_pages))
            r.shuffle(perm)
            for b, c in enumerate(cached):
                first, common = ref.member(b, groups, N, page, max_len, self.mp)
                for j in range(ref.entries(c, k, N, page)):
                    self.table[k][b][j] = self.table[k][first][j] if j < common else perm.pop()
                    if r.random() < bad:
                        self.table[k][b][j] = r.choice((-1, self.num_pages, 2 ** 31 - 1))
            self.count.append(min(len(perm), spare))
            self.free.append(perm[:self.count[-1]] + [-9] * (self.num_pages - self.count[-1]))
        # rows of a wider buffer, ranks and requests in it at other strides than a dense table's
        buf = torch.full((N, self.B + 1, self.mp + 3), -7, dtype=torch.int32, device=DEV)
        self.buf, self.t = buf, buf[:, :self.B, :self.mp]
        if self.B:
            self.t.copy_(ints(self.table).view(N, self.B, self.mp))
        self.f = torch.full((N, self.num_pages + 2), -9, dtype=torch.int32, device=DEV)[:, :self.num_pages]
        self.f.copy_(ints(self.free))
        self.c = ints(self.count)
        self.g = (None, None) if groups is None else (ints(groups[0]), ints(groups[1]))

    def reserve(self, new, T, inplace=False, arrays=True, stream=None):
        N, B = self.N, self.B
        x = dict(query_start=ints([-3] * (B + 1)), seq_lens=ints([-3] * B), missing=ints([-3] * N),
                 free_count=self.c if inplace else ints([-3] * N))
        if arrays:
            x.update(positions=ints([-3] * T), requests=ints([-3] * T), slots=ints([-3] * T, torch.int64))
        binding.page_reserve(ints(self.cached), ints(new), self.max_len, T, self.num_pages, self.page, self.t, self.f,
                             self.c, x["free_count"], x["missing"], x["query_start"], x["seq_lens"],
                             positions=x.get("positions"), slots=x.get("slots"), requests=x.get("requests"),
                             group_start=self.g[0], prefix_lens=self.g[1], stream=stream)
        return x

    def expect(self, new, T):
        return ref.reserve(self.cached, new, self.max_len, T, self.num_pages, self.page, self.table, self.free,
                           self.count, self.groups)


def compare(x, want, s, T):
    for name in ("query_start", "seq_lens", "missing", "free_count"):
        assert x[name].tolist() == want[name], name
    for name in ("positions", "requests", "slots"):
        if name in x:
            assert x[name].tolist() == want[name] + [-3] * (T - len(want[name])), name
    assert s.t.tolist() == want["block_table"]
    assert (s.buf[:, s.B:] == -7).all() and (s.buf[:, :, s.mp:] == -7).all()
    assert s.f.tolist() == s.free


def batch(B, N, page, max_len, q, seed, groups):
    r = random.Random(seed)
    cuts, plen, gr = None, None, None
    if groups:
        cuts = sorted(r.choice((0, 1, r.randrange(B + 1))) for _ in range(groups + 1))
        plen = [r.choice((0, 1, N * page - 1, N * page, r.randrange(max_len + 1), max_len)) for _ in range(groups)]
        gr = (cuts, plen)
    unit = N * page
    cached = []
    for b in range(B):
        first, common = ref.member(b, gr, N, page, max_len, 1 << 30)
        low = common * unit if first != b else (max([plen[g] for g in range(groups) if cuts[g] == b < cuts[g + 1]] + [0])
                                                if groups else 0)
        cached.append(r.choice((low, min(low + 1, max_len), r.randint(low, max_len), max_len)))
    new = [r.choice((0, 1, 1, r.randint(0, q), q)) for _ in range(B)]
    return cached, new, gr


CASES = [(B, N, page, max_len, q, groups) for B, N, page, max_len, q, groups in (
    (1, 1, 16, 100, 1, 0), (1, 3, 1, 33, 40, 0), (7, 2, 16, 300, 5, 2), (64, 4, 64, 3000, 1, 1), (33, 8, 8, 500, 70, 4),
    (9, 5, 128, 4000, 900, 3), (1023, 2, 16, 90, 3, 9), (1024, 3, 4, 40, 2, 0), (1025, 1, 2, 30, 7, 17),
    (2600, 2, 8, 64, 2, 70), (17, 16, 32, 2000, 33, 5), (3, 1, 65536, 200000, 1000, 1), (513, 9, 16, 600, 5, 3), (9000, 1, 8, 50, 2, 40),
    (8193, 2, 4, 20, 1, 1100))]


@pytest.mark.parametrize("B,N,page,max_len,q,groups", CASES)
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(B, N, page, max_len, q, groups, seed):
    cached, new, gr = batch(B, N, page, max_len, q, seed, groups)
    s = State(cached, N, page, max_len, gr, seed, wide=seed)
    T = sum(new) + 3 * seed
    want = s.expect(new, T)
    compare(s.reserve(new, T, inplace=bool(seed)), want, s, T)


def test_what_does_not_fit_is_cut_off():
    s = State([5, 90, 100, 0, 7], 2, 8, 100)
    for new, T in (([4, 50, 3, -6, 2], 40), ([4, 50, 3, 9, 2], 10), ([2 ** 31 - 1] * 5, 64), ([0] * 5, 0), ([-1] * 5, 7)):
        s2 = State(s.cached, 2, 8, 100)
        want = s2.expect(new, T)
        compare(s2.reserve(new, T), want, s2, T)


@pytest.mark.parametrize("spare", [0, 1, 5])
def test_empty_stacks(spare):
    cached, new, gr = batch(40, 3, 4, 200, 30, 5, 3)
    s = State(cached, 3, 4, 200, gr, spare=spare)
    want = s.expect(new, sum(new))
    assert sum(want["missing"]) > 0
    compare(s.reserve(new, sum(new)), want, s, sum(new))


def test_without_token_arrays_and_without_new_tokens():
    s = State([30, 17, 60], 2, 4, 64, ([0, 2], [16]))
    want = s.expect([3, 9, 4], 16)
    x = s.reserve([3, 9, 4], 16, arrays=False)
    compare(x, want, s, 16)
    s = State([64, 64, 64], 2, 4, 64, ([0, 3], [64]))
    want = s.expect([0, 0, 0], 0)
    compare(s.reserve([0, 0, 0], 0), want, s, 0)


def test_first_request_brings_the_prefix_in_the_same_call():
    # members hold nothing but the common pages, which the first request gets in this call
    s = State([0, 32, 32, 0], 2, 4, 100, ([0, 3], [35]))
    for k in range(2):
        for b in (1, 2):
            for j in range(4):
                s.table[k][b][j] = -7
    s.t.copy_(ints(s.table))
    new = [36, 5, 6, 40]
    want = s.expect(new, 90)
    assert want["block_table"][0][1][:4] == want["block_table"][0][0][:4] != [-7] * 4
    compare(s.reserve(new, 90), want, s, 90)


def test_members_that_hold_less_than_the_common_pages():
    # allowed: their tokens lie in the common pages then
    s = State([40, 3, 0], 2, 4, 100, ([0, 3], [40]))
    new = [1, 10, 50]
    want = s.expect(new, 61)
    compare(s.reserve(new, 61), want, s, 61)


@pytest.mark.parametrize("gs,pl", [([0, 0, 0], [9, 9]), ([2, 2, 3], [20, 20]), ([1, 3, 9], [30, 16]), ([-5, 2, 3], [50, 8]),
                                   ([0, 3], [2 ** 31 - 1]), ([0, 3], [-4])])
def test_odd_groups(gs, pl):
    # empty groups, one that reaches past the batch, one that begins before it, prefixes out of range
    B, N, page, max_len = 5, 2, 4, 64
    s = State([60] * B, N, page, max_len, (gs, pl))
    want = s.expect([2] * B, 10)
    if gs[0] < 0:                        # a group that begins before the batch is none
        s2 = State([60] * B, N, page, max_len, None)
        s.table, s.free, s.count, s.num_pages = s2.table, s2.free, s2.count, s2.num_pages
        s.t.copy_(ints(s.table))
        s.f = ints(s.free)
        s.c = ints(s.count)
        s.groups = ([2, 2, 3], pl)
        want = s.expect([2] * B, 10)
    compare(s.reserve([2] * B, 10), want, s, 10)


RELEASE = [(B, N, page, max_len, groups, bad) for B, N, page, max_len, groups, bad in (
    (1, 1, 16, 100, 0, 0.0), (5, 3, 1, 70, 2, 0.3), (64, 4, 64, 3000, 1, 0.0), (33, 8, 8, 500, 4, 0.1),
    (2047, 2, 8, 64, 9, 0.05), (2048, 1, 4, 40, 0, 0.0), (4500, 2, 16, 90, 31, 0.2), (3, 2, 2, 9000, 1, 0.01), (20, 1, 1, 3000, 2, 0.02), (16390, 1, 4, 20, 3, 0.1))]


@pytest.mark.parametrize("B,N,page,max_len,groups,bad", RELEASE)
@pytest.mark.parametrize("seed", [0, 1])
def test_release(B, N, page, max_len, groups, bad, seed):
    lens, _, gr = batch(B, N, page, max_len, 1, seed, groups)
    s = State(lens, N, page, max_len, gr, seed, spare=20, bad=bad)
    r = random.Random(seed)
    keep = [r.choice((-1, 0, 0, r.randrange(max_len), max_len + 5, l)) for l in lens]
    want = ref.release(lens, keep, max_len, s.num_pages, page, s.table, s.free, s.count, gr)
    out = s.c if seed else ints([-3] * N)
    lens_out = ints([-3] * B)
    binding.page_release(ints(lens), ints(keep), max_len, s.num_pages, page, s.t, s.f, s.c, out, lens_out=lens_out,
                         group_start=s.g[0], prefix_lens=s.g[1])
    assert out.tolist() == want["free_count"]
    assert s.f.tolist() == want["free_pages"]
    assert lens_out.tolist() == want["lens_out"]
    assert s.t.tolist() == s.table


def test_pages_beyond_the_capacity_are_dropped():
    s = State([64, 64], 2, 4, 64, spare=3)
    f, out = ints([[1, 2, 3, -9, -9]] * 2), ints([-3] * 2)
    want = ref.release([64, 64], [0, 8], 64, s.num_pages, 4, s.table, f.tolist(), [3, 4])
    binding.page_release(ints([64, 64]), ints([0, 8]), 64, s.num_pages, 4, s.t, f, ints([3, 4]), out)
    assert out.tolist() == want["free_count"] == [5, 5]
    assert f.tolist() == want["free_pages"]


def test_captured_steps_follow_the_lengths():
    """A graph of one step, replayed while the requests grow; pages that end come back to the next."""
    N, page, max_len, B, T = 2, 4, 120, 6, 8
    s = State([0] * B, N, page, max_len, seed=3, spare=4000)
    cached, new = ints([0] * B), ints([1] * B)
    x = {k: ints([-3] * n) for k, n in (("query_start", B + 1), ("seq_lens", B), ("missing", N), ("positions", T),
                                        ("requests", T))}
    slots = ints([-3] * T, torch.int64)

    def step():
        binding.page_reserve(cached, new, max_len, T, s.num_pages, page, s.t, s.f, s.c, s.c, x["missing"],
                             x["query_start"], x["seq_lens"], positions=x["positions"], slots=slots,
                             requests=x["requests"])
        cached.copy_(x["seq_lens"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    lens, table, count = [1] * B, ref.reserve([0] * B, [1] * B, max_len, T, s.num_pages, page, s.table, s.free, s.count), None
    table, count = table["block_table"], table["free_count"]
    for k in range(70):
        now = [(k + b) % 3 for b in range(B)]
        new.copy_(ints(now))
        want = ref.reserve(lens, now, max_len, T, s.num_pages, page, table, s.free, count)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        lens, table, count = want["seq_lens"], want["block_table"], want["free_count"]
        assert x["seq_lens"].tolist() == lens and s.c.tolist() == count
        assert s.t.tolist() == table
        n = want["query_start"][-1]
        assert slots.tolist()[:n] == want["slots"] and x["positions"].tolist()[:n] == want["positions"]
    # all pages come back, none twice
    binding.page_release(x["seq_lens"], ints([0] * B), max_len, s.num_pages, page, s.t, s.f, s.c, s.c)
    assert s.c.tolist() == s.count
    for r in range(N):
        assert sorted(s.f[r].tolist()[:s.count[r]]) == sorted(s.free[r][:s.count[r]])


def test_refusals_of_the_torch_layer():
    s = State([5, 6], 2, 4, 20)
    a = dict(cached=ints([5, 6]), new=ints([1, 1]), fc=s.c, out=ints([0, 0]), mi=ints([0, 0]), qs=ints([0] * 3),
             sl=ints([0] * 2))

    def call(max_len=20, T=2, slots=None, gs=None, pl=None, t=None, **c):
        v = {**a, **c}
        binding.page_reserve(v["cached"], v["new"], max_len, T, s.num_pages, 4, s.t if t is None else t, s.f, v["fc"],
                             v["out"], v["mi"], v["qs"], v["sl"], slots=slots, group_start=gs, prefix_lens=pl)

    call()
    for bad in (dict(cached=ints([5, 6], torch.int64)), dict(new=ints([1])), dict(qs=ints([0, 0])), dict(gs=ints([0, 1])),
                dict(pl=ints([3])), dict(gs=ints([0, 1, 2]), pl=ints([3])), dict(slots=ints([0, 0])),
                dict(max_len=1 << 31), dict(T=1 << 33), dict(cached=torch.tensor([5, 6], dtype=torch.int32)),
                dict(t=s.t.to(torch.int64))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(binding.DcpError):
        call(max_len=10 ** 6)
    with pytest.raises(binding.DcpError):
        call(sl=a["cached"])
