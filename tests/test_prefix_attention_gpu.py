"""Attention of batches whose requests share prefixes, against attention in 64
bits over every request's tokens: groups of every kind, prefixes that end inside a
page or are longer than a request, common parts that are cut over many CTAs, both
kernels, values that are not finite, padding, strides."""
import math

import pytest
import torch

from chunk_ref import DEV, Batch, assert_within, attention, share
from decode_context_attention_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


class Shared(Batch):
    """groups: [(first request, behind the last, common tokens), ...].  Members' tables name the first request's pages
    for the whole pages of the prefix, and their own, with the same rows, for the rest of it."""

    def __init__(self, lens, groups, own_entries="first", **kw):
        self.groups, self.own_entries = groups, own_entries
        super().__init__(lens, **kw)
        starts = [g[0] for g in groups] + [groups[-1][1]] if groups else [0]
        self.group_start = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.prefix_lens = torch.tensor([g[2] for g in groups], dtype=torch.int32, device=DEV)

    def fill(self):
        for lo, hi, n in self.groups:
            for b in range(lo + 1, min(hi, self.B)):
                m = min(n, len(self.k[b]), len(self.k[lo]))
                self.k[b][:m], self.v[b][:m] = self.k[lo][:m], self.v[lo][:m]
        super().fill()
        for lo, hi, n in self.groups:
            for b in range(lo + 1, min(hi, self.B)):
                # a page that the first request has not filled holds nothing of what follows for the others
                e = min(n, self.lens[lo][1], self.lens[b][1]) // self.N // self.page
                for r in range(self.N):
                    if self.own_entries == "first":
                        self.block_table[r, b, :e] = self.block_table[r, lo, :e]
                    elif self.own_entries == "bad":      # no pages at all
                        self.block_table[r, b, :e] = -5

    def scores(self, b, r, h):
        # the bound is a sum of magnitudes times that of the scale, which may be negative here
        s, err = super().scores(b, r, h)
        return s, err.abs()

    def outputs(self):
        o = torch.full((self.N, self.T, self.H, self.D), 7.0, dtype=self.dtype, device=DEV)
        return o, torch.full((self.N, self.T, self.H), 7.0, device=DEV)

    def run(self, causal=True, base="e", workspace=None, out=None, scale=None, stream=None):
        o, lse = out or self.outputs()
        binding.prefix_attention_paged(self.q, self.k_pages, self.v_pages, self.block_table, self.query_start,
                                       self.seq_lens, self.max_len, self.group_start, self.prefix_lens, o, lse,
                                       self.scale if scale is None else scale, base=base, causal=causal,
                                       workspace=workspace, stream=stream)
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        return o, lse

    def check(self, o, lse, causal=True, base="e"):
        want, z, o_tol, z_tol = attention(self, causal)
        n = self.start[-1]
        assert (o[:, n:] == 7.0).all() and (lse[:, n:] == 7.0).all()
        lse = lse * math.log(2.0) if base == "2" else lse
        assert_within(o[:, :n], want[:, :n], o_tol[:, :n], "o")
        assert_within(lse[:, :n], z[:, :n], z_tol[:, :n] + (2.0 ** -23 * z[:, :n].nan_to_num(0, 0, 0).abs()
                                                            if base == "2" else 0), "lse")


# lens, groups, arguments
CASES = {
    "two share, one token each": ([(1, 40), (1, 50)], [(0, 2, 32)], {}),
    "alone in its group": ([(1, 40), (3, 50), (1, 9)], [(0, 1, 32), (1, 2, 48)], {}),
    "no whole page": ([(1, 40), (1, 50)], [(0, 2, 31)], {}),
    "ends inside a page": ([(1, 90), (2, 80), (1, 77)], [(0, 3, 75)], {}),
    "loose requests around": ([(2, 30), (1, 70), (1, 66), (1, 80), (4, 20)], [(1, 4, 64)], {}),
    "three groups": ([(1, 70), (1, 66), (1, 40), (1, 45), (5, 200), (1, 199), (3, 198)],
                     [(0, 2, 64), (2, 4, 40), (4, 7, 190)], {}),
    "a holder without new tokens": ([(0, 64), (1, 70), (1, 65), (0, 64)], [(0, 4, 64)], {}),
    "nobody asks": ([(0, 64), (0, 70)], [(0, 2, 64)], {"pad": 2}),
    "one request asks": ([(0, 64), (1, 70)], [(0, 2, 64)], {}),
    "nothing behind the prefix but the new token": ([(1, 65), (1, 65), (1, 65)], [(0, 3, 64)], {}),
    "a request shorter than the prefix": ([(1, 200), (1, 40), (2, 220)], [(0, 3, 192)], {}),
    "a request of new tokens only": ([(1, 200), (40, 40), (2, 220)], [(0, 3, 192)], {}),
    "more new tokens than tokens": ([(1, 100), (9, 4), (1, 100)], [(0, 3, 96)], {}),
    "a prefix beyond every length": ([(1, 100), (1, 90)], [(0, 2, 10 ** 6)], {"max_len": 128}),
    "one rank": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"N": 1}),
    "three ranks": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"N": 3}),
    "eight ranks": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"N": 8, "page": 8}),
    "wide head dimension": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"D": 256}),
    "narrow head dimension": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"D": 64}),
    "pages of four": ([(1, 100), (3, 90), (1, 80)], [(0, 3, 77)], {"page": 4}),
    "pages of 256": ([(1, 1300), (3, 1290), (1, 1280)], [(0, 3, 1270)], {"page": 256}),
    "a head each": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"H": 3, "Hkv": 3}),
    "twelve heads a group": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"H": 24, "Hkv": 2}),
    "five heads a group": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"H": 5, "Hkv": 1}),
    "64 heads a group": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"H": 64, "Hkv": 1}),
    "padding and strides": ([(1, 300), (3, 290), (1, 280)], [(0, 3, 270)], {"pad": 3, "strided": True}),
    "more than a block of rows": ([(1, 70 + b % 9) for b in range(150)], [(0, 150, 64)], {"H": 4, "Hkv": 2}),
    "chunks": ([(150, 420), (90, 380), (133, 500), (1, 300)], [(0, 4, 290)], {}),
    # groups of enough requests and tokens for a common part of their own
    "many": ([(1, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {}),
    "many, drafts": ([(1 + b % 4, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {}),
    "many, of two and of three row blocks": ([(b % 3 + 6, 700 + 3 * b) for b in range(12)], [(0, 12, 690)], {}),
    "many, of four row blocks": ([(9 + b % 8, 700 + 3 * b) for b in range(12)], [(0, 12, 640)], {}),
    "many, and wide ones": ([(1 + 16 * (b % 2), 1700 + 3 * b) for b in range(12)], [(0, 12, 1660)], {}),
    "many, all wide": ([(17 + b, 2100 + 3 * b) for b in range(9)], [(0, 9, 2048)], {}),
    "many, one rank": ([(1, 500 + 3 * b) for b in range(20)], [(0, 20, 490)], {"N": 1}),
    "many, three ranks, loose ones": ([(1, 30)] + [(2, 900 + 3 * b) for b in range(20)] + [(1, 800), (70, 200)],
                                      [(1, 21, 890)], {"N": 3}),
    "many, D 64": ([(1 + b % 3, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {"D": 64}),
    "many, D 256": ([(1 + b % 3, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {"D": 256}),
    "many, D 256, 32 rows and more": ([(7 + b % 3, 900 + 3 * b) for b in range(14)], [(0, 14, 890)], {"D": 256}),
    "many, D 256, cut": ([(1, 4100 + b) for b in range(8)], [(0, 8, 4096)], {"D": 256, "N": 1, "H": 4, "Hkv": 1}),
    "many, a head each": ([(1 + b % 5, 900 + 3 * b) for b in range(20)], [(0, 20, 880)], {"H": 3, "Hkv": 3}),
    "many, 64 tokens of a head each": ([(60 + b % 5, 1900 + 3 * b) for b in range(12)], [(0, 12, 1700)],
                                       {"H": 2, "Hkv": 2, "N": 1}),
    "many, five heads a group": ([(1 + b % 3, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {"H": 5, "Hkv": 1}),
    "many, 64 heads a group": ([(1, 700 + 3 * b) for b in range(12)], [(0, 12, 690)], {"H": 64, "Hkv": 1}),
    "many, pages of four": ([(1 + b % 2, 700 + 3 * b) for b in range(20)], [(0, 20, 690)], {"page": 4}),
    "many, pages of one": ([(1 + b % 2, 400 + 3 * b) for b in range(20)], [(0, 20, 390)], {"page": 1, "Hkv": 1}),
    "many, pages of 512": ([(1, 2500 + 3 * b) for b in range(12)], [(0, 12, 2490)], {"page": 512}),
    "many, padding and strides": ([(1 + b % 3, 700 + 3 * b) for b in range(20)], [(0, 20, 690)],
                                  {"pad": 3, "strided": True}),
    "many, three groups": ([(1, 900 + 3 * b) for b in range(12)] + [(2, 640 + b) for b in range(14)]
                           + [(1, 2000 + b) for b in range(10)], [(0, 12, 890), (12, 26, 512), (26, 36, 1999)], {}),
    "many, a holder": ([(0, 768)] + [(1, 770 + 3 * b) for b in range(20)], [(0, 21, 768)], {}),
    "many, cut over many CTAs": ([(1, 12100 + b) for b in range(9)], [(0, 9, 12000)],
                                 {"H": 2, "Hkv": 1, "page": 64}),
    "many, long own parts": ([(1, 700 + 900 * b) for b in range(9)], [(0, 9, 640)], {"H": 4, "Hkv": 1, "page": 64}),
    "many, one shorter": ([(1, 900 + 3 * b) for b in range(19)] + [(1, 500)], [(0, 20, 880)], {}),
    "cut over many CTAs": ([(1, 12100), (1, 12050), (2, 12033)], [(0, 3, 12000)], {"H": 2, "Hkv": 1, "page": 64}),
    "cut, wide": ([(1, 9100), (1, 9050), (2, 9033)], [(0, 3, 9000)], {"H": 2, "Hkv": 1, "page": 64, "D": 256, "N": 1}),
    "own parts cut": ([(1, 9100), (1, 7050), (2, 8033)], [(0, 3, 128)], {"H": 2, "Hkv": 1, "page": 64, "N": 1}),
    "loose and cut": ([(1, 9100), (1, 500), (2, 433), (1, 9000)], [(1, 3, 400)], {"H": 2, "Hkv": 1, "page": 64, "N": 1}),
}


# the same behind prefixes that are longer by more than the tokens of a rank up to which a batch counts as small
for name in [n for n in CASES if n.startswith("many")]:
    lens, groups, kw = CASES[name]
    more = 1040 * kw.get("N", 2)
    inside = {b for lo, hi, n in groups for b in range(lo, hi)}
    CASES[name.replace("many", "many, long")] = (
        [(n, l + more if b in inside else l) for b, (n, l) in enumerate(lens)], [(lo, hi, n + more) for lo, hi, n in groups],
        kw)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_shared_prefixes(name, dtype):
    lens, groups, kw = CASES[name]
    bt = Shared(lens, groups, dtype=dtype, seed=len(name), **kw)
    o, lse = bt.run()
    bt.check(o, lse)


@pytest.mark.parametrize("name", ["three groups", "a request shorter than the prefix", "a request of new tokens only",
                                  "more new tokens than tokens", "chunks", "wide head dimension", "many, drafts",
                                  "many, and wide ones", "many, D 256", "many, three ranks, loose ones",
                                  "many, one shorter", "many, long, drafts", "many, long, and wide ones",
                                  "many, long, D 256", "many, long, three ranks, loose ones", "many, long, one shorter"])
def test_not_causal_and_base_2(name):
    lens, groups, kw = CASES[name]
    bt = Shared(lens, groups, seed=5, **kw)
    o, lse = bt.run(causal=False, base="2")
    bt.check(o, lse, causal=False, base="2")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q", [1, 40])
def test_a_large_groups_prefix_is_read_once(D, q):
    """Members whose tables name no pages for the common part: only the first request's entries can have been read."""
    n = 2200 if q == 1 else 6400      # (less is done sooner by each request on its own)
    bt = Shared([(q if b < 24 else 1, n + 50 + 2 * b) for b in range(30)], [(0, 30, n)], own_entries="bad", D=D, H=4,
                Hkv=2)
    o, lse = bt.run()
    bt.check(o, lse)


@pytest.mark.parametrize("D", [64, 256])
def test_negative_scale_and_large_scores(D):
    for scale, qs in ((-0.09, 1.0), (0.09, 60.0), (0.0, 1.0)):
        for lens, groups in (([(1, 200), (1, 190), (2, 180)], [(0, 3, 160)]),
                             ([(1 + b % 2, 700 + 3 * b) for b in range(20)], [(0, 20, 690)]),
                             ([(1 + b % 2, 2900 + 3 * b) for b in range(20)], [(0, 20, 2890)])):
            bt = Shared(lens, groups, D=D, qscale=qs, dtype=torch.float16)
            bt.scale = scale
            o, lse = bt.run(scale=scale)
            bt.check(o, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("where", ["prefix", "own", "future"])
@pytest.mark.parametrize("lens,n", [([(2, 200), (1, 190), (3, 180)], 160),
                                    ([(2, 740), (1, 735)] * 9 + [(3, 720)], 690),
                                    ([(2, 2940), (1, 2935)] * 9 + [(3, 2920)], 2890),
                                    ([(2, 740), (1, 735)] * 9 + [(50, 720)], 660)])
def test_values_that_are_not_finite(D, where, lens, n):
    bt = Shared(lens, [(0, len(lens), n)], D=D, dtype=torch.float16, N=2)
    last = lens[-1][1]
    g = {"prefix": 7, "own": n + 5, "future": last - 1}[where]
    x = math.inf if where != "own" else math.nan
    for b in range(len(lens)) if where == "prefix" else (len(lens) - 1,):
        bt.v[b][g, 1, 5] = x
    bt.fill()
    o, lse = bt.run()
    bt.check(o, lse)


@pytest.mark.parametrize("D", [128, 256])
def test_equal_calls_give_equal_bits_and_padding_changes_none(D):
    lens, groups = [(1, 2900 + 7 * b) for b in range(20)] + [(40, 900)], [(0, 12, 2840), (12, 21, 300)]
    bt = Shared(lens, groups, pad=4, D=D)
    o, lse = bt.run()
    ws = torch.full((binding.prefix_workspace_bytes(bt.N, bt.B, bt.T, bt.H, bt.Hkv, D, bt.max_len, 2),), 255,
                    dtype=torch.uint8, device=DEV)
    bt.q[-4:] = math.nan
    o2, lse2 = bt.run(workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_without_groups_it_is_the_extend():
    lens = [(1, 700), (3, 90), (40, 400), (0, 5)]
    bt = Shared(lens, [])
    o, lse = bt.outputs()
    binding.extend_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len,
                                   o, lse, bt.scale)
    o1, lse1 = bt.run()
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    bt.group_start = bt.prefix_lens = None
    o1, lse1 = bt.run()
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    # groups that share nothing: the same parts, written by the kernel itself or joined
    bt = Shared(lens, [(0, 1, 64), (1, 4, 0)])
    o1, lse1 = bt.run()
    bt.check(o1, lse1)


@pytest.mark.parametrize("gs,pl", [([0, 0, 3], [99, 96]), ([3, 3, 3], [96, 96]), ([0, 2, 7], [96, 96]),
                                   ([-4, 2, 3], [96, 96]), ([2, 0, 3], [96, 96]), ([0, 3, 1], [96, 2 ** 31 - 1]),
                                   ([0, 1, 3], [-3, -2 ** 31])])
@pytest.mark.parametrize("D", [128, 256])
def test_odd_groups_stay_in_bounds(gs, pl, D):
    """Empty groups, groups that reach out of the batch, borders out of order: what is documented is checked, the rest
    ends without touching anything else."""
    bt = Shared([(1, 200), (1, 190), (2, 180)], [(0, 3, 96)], D=D)
    bt.group_start = torch.tensor(gs, dtype=torch.int32, device=DEV)
    bt.prefix_lens = torch.tensor(pl, dtype=torch.int32, device=DEV)
    o, lse = bt.run()
    if gs == sorted(gs):
        bt.check(o, lse)


def test_captured_while_lengths_and_groups_change():
    """One graph; the batch's arrays change between replays, its workspace is its own."""
    big = [(1, 700), (1, 690), (1, 650), (1, 720), (2, 600)]
    bt = Shared(big, [(0, 3, 600), (3, 5, 512)], pad=3, max_len=800)
    out = bt.outputs()
    ws = torch.empty(binding.prefix_workspace_bytes(bt.N, bt.B, bt.T, bt.H, bt.Hkv, bt.D, bt.max_len, 2),
                     dtype=torch.uint8, device=DEV)
    call = None
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call = binding.prepare_prefix_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start,
                                                      bt.seq_lens, bt.max_len, bt.group_start, bt.prefix_lens, *out,
                                                      bt.scale, workspace=ws)
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call2 = binding.prepare_prefix_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start,
                                                           bt.seq_lens, bt.max_len, bt.group_start, bt.prefix_lens, *out,
                                                           bt.scale, workspace=ws)
            call2()
    for lens, groups in ((big, [(0, 3, 600), (3, 5, 512)]), ([(1, 790), (1, 780), (1, 770), (1, 765), (1, 760)],
                                                              [(0, 5, 750), (5, 5, 0)]),
                         ([(2, 300), (1, 256), (0, 100), (1, 90), (4, 400)], [(0, 2, 256), (2, 5, 64)]),
                         ([(1, 10), (1, 20), (1, 5), (1, 1), (1, 3)], [(0, 5, 700), (5, 5, 9)])):
        x = Shared(lens, groups, max_len=800, pad=bt.T - sum(n for n, _ in lens), seed=8)
        x.num_pages = x.k_pages.shape[1]
        assert x.k_pages.shape == bt.k_pages.shape and x.block_table.shape == bt.block_table.shape
        for name in ("q", "k_pages", "v_pages", "block_table", "query_start", "seq_lens", "group_start", "prefix_lens"):
            getattr(bt, name).copy_(getattr(x, name))
        for t in out:
            t.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        x.check(*out)


# on both sides of what counts as a small batch: tokens of a rank, rows of a request, tiles in all, requests
EDGES = {
    "1024 tokens of a rank": ([(1, 1024)] * 3 + [(1, 900)], [(0, 4, 880)], {"N": 1}),
    "1025 tokens of a rank": ([(1, 1024)] * 3 + [(1, 1025)], [(0, 4, 880)], {"N": 1}),
    "1025 tokens of the second rank's": ([(1, 2048), (1, 2049)] * 2, [(0, 4, 1900)], {"N": 2}),
    "rows of four warps": ([(8, 300), (8, 310), (1, 290)], [(0, 3, 270)], {"H": 8, "Hkv": 1}),
    "a row more": ([(8, 300), (9, 310), (1, 290)], [(0, 3, 270)], {"H": 8, "Hkv": 1}),
    "1900 tiles": ([(1, 1024 - 128 * 4 - 20)] * 25, [(0, 25, 480)], {"N": 1, "H": 19, "Hkv": 19, "D": 64, "page": 8}),
    "more than 1900 tiles": ([(1, 1024 - 128 * 4 - 20)] * 26, [(0, 26, 480)],
                             {"N": 1, "H": 19, "Hkv": 19, "D": 64, "page": 8}),
    "D 256, half of them": ([(1, 500)] * 12 + [(1, 100)], [(0, 12, 480)],
                            {"N": 1, "H": 19, "Hkv": 19, "D": 256, "page": 8}),
    "4096 places": ([(1, 110 + b // 100) if b % 400 == 0 else (0, 0) for b in range(4096)], [(0, 4096, 96)], {"N": 1}),
    "4097 places": ([(1, 110 + b // 100) if b % 400 == 0 else (0, 0) for b in range(4097)], [(0, 4097, 96)], {"N": 1}),
}


@pytest.mark.parametrize("name", EDGES)
def test_edges_of_small_batches(name):
    lens, groups, kw = EDGES[name]
    bt = Shared(lens, groups, seed=len(name), **kw)
    bt.check(*bt.run())


def test_captured_while_a_batch_grows_out_of_being_small():
    """One graph, one workspace: replays whose batch the last kernel does alone, and such that share, in turn."""
    N = 2
    of = lambda n, own, q: ([(1 + (b + q) % 2, n + own + 3 * b) for b in range(12)], [(0, 12, n)])
    big, small = of(2400, 90, 0), of(300, 70, 1)
    bt = Shared(*big, pad=2, max_len=2700)
    out = bt.outputs()
    ws = torch.full((binding.prefix_workspace_bytes(N, bt.B, bt.T, bt.H, bt.Hkv, bt.D, bt.max_len, 1),), 255,
                    dtype=torch.uint8, device=DEV)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call = binding.prepare_prefix_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start,
                                                      bt.seq_lens, bt.max_len, bt.group_start, bt.prefix_lens, *out,
                                                      bt.scale, workspace=ws)
        with torch.cuda.graph(graph, stream=side):
            call()
    for k, (lens, groups) in enumerate((small, big, big, small, of(1500, 40, 1), small, of(2048, 200, 0))):
        x = Shared(lens, groups, max_len=2700, pad=bt.T - sum(n for n, _ in lens), seed=20 + k)
        assert x.k_pages.shape == bt.k_pages.shape and x.block_table.shape == bt.block_table.shape
        for name in ("q", "k_pages", "v_pages", "block_table", "query_start", "seq_lens", "group_start", "prefix_lens"):
            getattr(bt, name).copy_(getattr(x, name))
        for t in out:
            t.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        x.check(*out)


def test_two_calls_at_once_on_their_own_workspaces():
    a = Shared([(1, 900 + b) for b in range(30)], [(0, 30, 880)], seed=1)
    b = Shared([(1, 700 + b) for b in range(9)] + [(50, 800)], [(0, 9, 640)], D=64, dtype=torch.float16, seed=2)
    outs = [a.outputs(), b.outputs()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, out, s in zip((a, b), outs, streams):
            binding.prefix_attention_paged(x.q, x.k_pages, x.v_pages, x.block_table, x.query_start, x.seq_lens,
                                           x.max_len, x.group_start, x.prefix_lens, *out, x.scale, stream=s)
    torch.cuda.synchronize()
    for x, out in zip((a, b), outs):
        x.check(*out)


def test_refusals_of_the_torch_layer():
    bt = Shared([(1, 40), (1, 50)], [(0, 2, 32)])
    good = bt.group_start, bt.prefix_lens
    for gs, pl in ((good[0], None), (None, good[1]), (good[0][:1], good[1]), (good[0].long(), good[1]),
                   (good[0].cpu(), good[1].cpu()), (good[0], good[1].float())):
        bt.group_start, bt.prefix_lens = gs, pl
        with pytest.raises(ValueError):
            bt.run()
    bt.group_start, bt.prefix_lens = good
    with pytest.raises(binding.DcpError):      # a workspace that the extend alone would take
        bt.run(workspace=torch.empty(binding.extend_workspace_bytes(bt.N, bt.B, bt.T, bt.H, bt.Hkv, bt.D, bt.max_len),
                                     dtype=torch.uint8, device=DEV))
