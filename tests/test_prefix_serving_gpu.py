"""Page bookkeeping and shared prefixes as a server uses them: requests join groups
behind a prefix that one request holds, bring tokens, decode, end, and their pages go
to others; a step is pages and index arrays from lengths, the append, the attention
and the merge, eager or one graph.  Every output against attention in 64 bits over the
tokens that the requests were given, every cache row against what was appended, and all
pages back at the end.  The same from two threads, and with loads that never come."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Serving:
    """Requests 0..4 share their first 150 tokens, which 0 holds, 5..11 their first 333, which 5 holds; 12 and 13 are on
    their own."""
    B, T, GROUPS, PREFIX = 14, 700, [0, 5, 12], [150, 333]

    def __init__(self, N=2, H=8, Hkv=2, D=128, page=16, max_len=800, dtype=torch.bfloat16, seed=0):
        self.N, self.H, self.Hkv, self.D, self.page, self.max_len, self.dtype = N, H, Hkv, D, page, max_len, dtype
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        B, T = self.B, self.T
        mp = -(-(-(-max_len // N)) // page)
        self.num_pages = B * mp
        perm = torch.stack([torch.randperm(self.num_pages, generator=self.g, device=DEV) for _ in range(N)]).int()
        self.free, self.count = perm.contiguous(), ints([self.num_pages] * N)
        self.k_pages = torch.full((N, self.num_pages, page, Hkv, D), math.nan, dtype=dtype, device=DEV)
        self.v_pages = torch.full_like(self.k_pages, math.nan)
        self.table = torch.full((N, B, mp), -1, dtype=torch.int32, device=DEV)
        self.cached, self.new, self.missing = ints([0] * B), ints([0] * B), ints([0] * N)
        self.qs, self.sl, self.pos, self.req = ints([0] * (B + 1)), ints([0] * B), ints([-1] * T), ints([-1] * T)
        self.slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
        self.gs, self.pl = ints(self.GROUPS), ints(self.PREFIX)
        self.q, self.qn = (torch.zeros((T, H, D), dtype=dtype, device=DEV) for _ in range(2))
        self.k, self.v = (torch.zeros((T, Hkv, D), dtype=dtype, device=DEV) for _ in range(2))
        self.o = torch.zeros((N, T, H, D), dtype=dtype, device=DEV)
        self.lse = torch.zeros((N, T, H), device=DEV)
        self.out, self.out_lse = torch.zeros((T, H, D), dtype=dtype, device=DEV), torch.zeros((T, H), device=DEV)
        self.scale = D ** -0.5
        self.ws = torch.empty(binding.prefix_workspace_bytes(N, B, T, H, Hkv, D, max_len, 2), dtype=torch.uint8, device=DEV)
        empty = torch.zeros((0, Hkv, D), dtype=dtype, device=DEV)
        self.has_k, self.has_v = [empty] * B, [empty] * B      # what every request was given
        self.graph = None
        torch.cuda.synchronize()

    def device_step(self):
        binding.page_reserve(self.cached, self.new, self.max_len, self.T, self.num_pages, self.page, self.table, self.free,
                             self.count, self.count, self.missing, self.qs, self.sl, positions=self.pos,
                             slots=self.slots, requests=self.req, group_start=self.gs, prefix_lens=self.pl)
        binding.qk_norm_rope_append(self.q, self.k, self.v, None, None, 0.0, None, None, self.k_pages, self.v_pages,
                                    self.table, self.qs, self.sl, self.max_len, self.qn)
        binding.prefix_attention_paged(self.qn, self.k_pages, self.v_pages, self.table, self.qs, self.sl, self.max_len,
                                       self.gs, self.pl, self.o, self.lse, self.scale, base="2", workspace=self.ws)
        binding.lse_combine(self.o, self.lse, self.out, self.out_lse, base="2")
        self.cached.copy_(self.sl)

    def capture(self):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.device_step()
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.device_step()
        torch.cuda.current_stream().wait_stream(side)

    def joins(self, b, holder, group):
        """Request b begins with the whole pages that `holder` has of the group's prefix; returns the rest of the
        prefix, which it brings itself."""
        unit = self.N * self.page
        n = self.PREFIX[group] // unit * unit
        self.has_k[b], self.has_v[b] = self.has_k[holder][:n], self.has_v[holder][:n]
        self.cached[b] = n
        rest = slice(n, self.PREFIX[group])
        return self.has_k[holder][rest], self.has_v[holder][rest]

    def step(self, new, given=None):
        """new[b] tokens for every request, the first ones of which are given[b] = (keys, values)."""
        T = sum(new)
        self.q.copy_((torch.randn((self.T, self.H, self.D), generator=self.g, device=DEV) * 1.5).to(self.dtype))
        self.k.copy_(torch.randn((self.T, self.Hkv, self.D), generator=self.g, device=DEV).to(self.dtype))
        self.v.copy_(torch.randn((self.T, self.Hkv, self.D), generator=self.g, device=DEV).to(self.dtype))
        start = [0]
        for b, n in enumerate(new):
            if given and b in given:
                k, v = given[b]
                self.k[start[-1]:start[-1] + len(k)], self.v[start[-1]:start[-1] + len(v)] = k, v
            start.append(start[-1] + n)
        self.new.copy_(ints(new))
        if self.graph is None:
            self.device_step()
        else:
            self.graph.replay()
        torch.cuda.synchronize()
        assert binding.device_status() == 0 and self.missing.tolist() == [0] * self.N
        assert self.qs.tolist() == start
        for b, n in enumerate(new):
            s = slice(start[b], start[b + 1])
            self.has_k[b] = torch.cat([self.has_k[b], self.k[s]])
            self.has_v[b] = torch.cat([self.has_v[b], self.v[s]])
        assert self.sl.tolist() == [len(x) for x in self.has_k]
        assert self.pos[:T].tolist() == [len(self.has_k[b]) - n + j for b, n in enumerate(new) for j in range(n)]
        assert self.req[:T].tolist() == [b for b, n in enumerate(new) for _ in range(n)]
        flat = self.k_pages.view(-1, self.Hkv, self.D)
        assert torch.equal(flat[self.slots[:T]], self.k[:T])
        u = U[self.dtype]
        for b, n in enumerate(new):
            if not n:
                continue
            s, L = slice(start[b], start[b + 1]), len(self.has_k[b])
            G = self.H // self.Hkv
            k, v = (x.double().repeat_interleave(G, 1) for x in (self.has_k[b], self.has_v[b]))
            x = torch.einsum("thd,lhd->htl", self.qn[s].double(), k) * self.scale
            seen = torch.arange(L, device=DEV)[None] <= (L - n + torch.arange(n, device=DEV))[:, None]
            x = torch.where(seen[None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            w = (x - z[..., None]).exp()
            want, mass = torch.einsum("htl,lhd->thd", w, v), torch.einsum("htl,lhd->thd", w, v.abs())
            # P, the partials and the merged output are rounded once each; 2^-10 covers the 32-bit arithmetic
            err = (self.out[s].double() - want).abs() - (2 * u + 2.0 ** -10) * mass - u * want.abs()
            assert err.max().item() <= 0, (b, err.max().item())
            assert (self.out_lse[s].double() - z.T / math.log(2.0)).abs().max().item() <= 1e-4

    def end(self, requests, groups=True):
        keep = [0 if b in requests else -1 for b in range(self.B)]
        left = ints([-1] * self.B)
        binding.page_release(self.cached, ints(keep), self.max_len, self.num_pages, self.page, self.table, self.free,
                             self.count, self.count, lens_out=left, group_start=self.gs if groups else None,
                             prefix_lens=self.pl if groups else None)
        self.cached.copy_(left)
        for b in requests:
            self.has_k[b], self.has_v[b] = self.has_k[b][:0], self.has_v[b][:0]

    def run(self, graph=False):
        B = self.B
        one = [1] * B
        # the holders bring the prefixes, a request on its own a prompt
        first = [0] * B
        first[0], first[5], first[12] = 150, 333, 90
        self.step(first)
        if graph:
            self.new.zero_()
            self.capture()
        # members join, two of them with more than the rest of the prefix
        given = {b: self.joins(b, 0, 0) for b in (1, 2, 3)} | {b: self.joins(b, 5, 1) for b in (6, 7, 8, 9, 10)}
        new = [0] * B
        for b in given:
            new[b] = len(given[b][0]) + (40 if b in (2, 7) else 1)
        self.step(new, given)
        one[0] = one[5] = one[4] = one[11] = one[13] = 0          # holders and empty places
        for _ in range(3):
            self.step(one)
        # drafts, single tokens and nothing in one step
        self.step([0, 3, 1, 4, 0, 0, 2, 1, 0, 4, 1, 0, 3, 77])
        # some end; others take their places and pages
        self.end([2, 8, 12])
        given = {2: self.joins(2, 0, 0), 4: self.joins(4, 0, 0), 8: self.joins(8, 5, 1), 11: self.joins(11, 5, 1)}
        new = [0, 1, len(given[2][0]) + 7, 1, len(given[4][0]) + 30, 0, 1, 1, len(given[8][0]) + 2, 1, 1,
               len(given[11][0]) + 64, 120, 1]
        self.step(new, given)
        for _ in range(2):
            self.step([0, 1, 1, 1, 1, 0, 1, 1, 1, 1, 1, 1, 1, 1])
        # the members first, then the holders, whose pages they had
        self.end([b for b in range(B) if b not in (0, 5)])
        self.end([0, 5], groups=False)
        assert self.count.tolist() == [self.num_pages] * self.N
        assert torch.equal(self.free.sort(-1).values, torch.arange(self.num_pages, device=DEV).int().expand_as(self.free))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kw", [dict(), dict(N=3, D=64, page=8, dtype=torch.float16), dict(N=1, H=4, Hkv=1, D=256),
                                dict(N=4, H=12, Hkv=1, page=32), dict(N=2, H=6, Hkv=6, D=64, page=4)])
def test_serving(kw, graph):
    Serving(**kw).run(graph)


def test_from_two_threads():
    errors = []

    def work(seed):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                Serving(seed=seed, N=1 + seed).run()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


STALL = r"""
import os, sys
sys.path[:0] = [sys.argv[1], os.path.join(sys.argv[1], "tests")]
import torch
from decode_context_attention_gb300 import binding
from test_prefix_attention_gpu import Shared
for D, page in ((64, 16), (128, 16), (256, 16)):
    for more in (0, 2200):
        bt = Shared([(1 + b % 2, more + 700 + 3 * b) for b in range(20)], [(0, 20, more + 690)], D=D, page=page)
        o, lse = bt.outputs()
        os.environ["DCP_TEST_STALL_LOADS"] = "1"
        binding.prefix_attention_paged(bt.q, bt.k_pages, bt.v_pages, bt.block_table, bt.query_start, bt.seq_lens, bt.max_len,
                                       bt.group_start, bt.prefix_lens, o, lse, bt.scale)
        torch.cuda.synchronize()
        assert binding.device_status() == 7, "expected DCP_ERR_TIMEOUT"
        assert binding.device_status() == 0, "the status must clear once read"
        del os.environ["DCP_TEST_STALL_LOADS"]
        bt.check(*bt.run())
print("timeouts reported, context usable")
"""


def test_waits_that_run_out_are_reported_and_leave_the_context_usable():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ)
    env.pop("DCP_TEST_STALL_LOADS", None)
    r = subprocess.run([sys.executable, "-c", STALL, root], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "timeouts reported, context usable" in r.stdout
