"""The chunk-serving operators as a server uses them: prompts appended and
attended in ragged chunks over N ranks, the partials merged, the weights
accumulated with the merged log-sum-exp, the caches evicted, single tokens
decoded over what is left; against attention in 64 bits over the tokens a step
sees.  The same captured into graphs, from two threads, and with loads that
never come."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from decode_context_attention_gb300 import binding, build

from chunk_ref import DEV, U, share

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    binding.load()


class Server:
    def __init__(self, N=3, B=3, H=8, Hkv=2, D=128, page=16, max_len=900, keep=64, dtype=torch.bfloat16, seed=0):
        self.N, self.B, self.H, self.Hkv, self.D, self.page, self.max_len, self.keep = N, B, H, Hkv, D, page, max_len, keep
        self.dtype = dtype
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.cap = -(-max_len // N)
        mp = -(-self.cap // page)
        kp = mp                                                # pages to move into
        pages = B * (mp + kp) + 2
        perm = torch.stack([torch.randperm(pages, generator=self.g, device=DEV) for _ in range(N)]).to(torch.int32)
        self.table = perm[:, : B * mp].reshape(N, B, mp).contiguous()
        self.spare = perm[:, B * mp: B * (mp + kp)].reshape(N, B, kp).contiguous()
        self.k_pages = torch.full((N, pages, page, Hkv, D), math.nan, dtype=dtype, device=DEV)
        self.v_pages = torch.full_like(self.k_pages, math.nan)
        self.acc = torch.full((N, B, Hkv, self.cap), math.nan, device=DEV)
        ang = torch.arange(max_len + 8, device=DEV, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(D // 2, device=DEV, dtype=torch.float64) / (D // 2))
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], -1).float()
        self.qw, self.kw = ((1 + 0.1 * torch.randn(D, generator=self.g, device=DEV)).to(dtype) for _ in range(2))
        self.lens, self.seen = [0] * B, [0] * B                # tokens held; positions used
        # what every request's heads hold, by (rank, request, head): lists of (K row, V row), as read from the pages
        self.scale = D ** -0.5

    def batch(self, new, pad=0):
        T = sum(new) + pad
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        qkv = torch.randn((T, self.H + 2 * self.Hkv, self.D), generator=self.g, device=DEV).to(self.dtype)
        pos = [self.seen[b] + j for b, n in enumerate(new) for j in range(n)] + [0] * pad
        for b, n in enumerate(new):
            self.lens[b] += n
            self.seen[b] += n
        return dict(q=qkv[:, :self.H], k=qkv[:, self.H:self.H + self.Hkv], v=qkv[:, self.H + self.Hkv:],
                    pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
                    qs=torch.tensor(start, dtype=torch.int32, device=DEV),
                    sl=torch.tensor(self.lens, dtype=torch.int32, device=DEV), new=new, start=start, T=T,
                    qn=torch.zeros((T, self.H, self.D), dtype=self.dtype, device=DEV),
                    o=torch.zeros((self.N, T, self.H, self.D), dtype=self.dtype, device=DEV),
                    lse=torch.zeros((self.N, T, self.H), device=DEV),
                    out=torch.zeros((T, self.H, self.D), dtype=self.dtype, device=DEV),
                    out_lse=torch.zeros((T, self.H), device=DEV))

    def append(self, x):
        binding.qk_norm_rope_append(x["q"], x["k"], x["v"], self.qw, self.kw, 1e-6, self.cos_sin, x["pos"],
                                    self.k_pages, self.v_pages, self.table, x["qs"], x["sl"], self.max_len, x["qn"])

    def chunk(self, x, ws=None):
        self.append(x)
        binding.extend_attention_paged(x["qn"], self.k_pages, self.v_pages, self.table, x["qs"], x["sl"], self.max_len,
                                       x["o"], x["lse"], self.scale, base="2", workspace=ws)
        binding.lse_combine(x["o"], x["lse"], x["out"], x["out_lse"], base="2")
        binding.attention_weights_paged(x["qn"], self.k_pages, self.table, x["qs"], x["sl"], self.max_len, x["out_lse"],
                                        self.acc, self.scale, base="2")

    def decode(self, x, ws=None):
        self.append(x)
        binding.decode_attention_paged(x["qn"], self.k_pages, self.v_pages, self.table, x["sl"], self.max_len, x["o"],
                                       x["lse"], self.scale, base="2", split_tokens=128, workspace=ws)
        binding.lse_combine(x["o"], x["lse"], x["out"], x["out_lse"], base="2")

    def evict(self, keep, recent):
        kept = torch.full((self.N, self.B, self.Hkv, self.cap), -1, dtype=torch.int32, device=DEV)
        acc = torch.full_like(self.acc, math.nan)
        binding.cache_evict_paged(self.k_pages, self.v_pages, self.table,
                                  torch.tensor(self.lens, dtype=torch.int32, device=DEV), self.max_len, self.acc,
                                  torch.full((self.B,), keep, dtype=torch.int32, device=DEV), keep, recent, self.spare,
                                  kept, acc)
        self.table, self.spare, self.acc = self.spare, self.table, acc
        self.lens = [min(l, keep) for l in self.lens]
        return kept

    def held(self, r, b, h):
        """K and V of the local tokens of (rank, request, head), from the pages, in 64 bits."""
        i = torch.arange(share(self.lens[b], r, self.N), device=DEV)
        pg = self.table[r, b].long()[i // self.page]
        return (self.k_pages[r, pg, i % self.page, h].double(), self.v_pages[r, pg, i % self.page, h].double(), i)

    def expect(self, x, b, h):
        """Output, log-sum-exp (base 2) and weights by rank of request b's new tokens, attending everything visible."""
        n, s = x["new"][b], slice(x["start"][b], x["start"][b + 1])
        q = x["qn"][s, h].double()
        ks, vs, seen, ranks = [], [], [], []
        for r in range(self.N):
            k, v, i = self.held(r, b, h // (self.H // self.Hkv))
            g = self.lens[b] - n + torch.arange(n, device=DEV)
            ks.append(k), vs.append(v), ranks.append(len(i))
            seen.append((i * self.N + r)[None] <= g[:, None])
        k, v, seen = torch.cat(ks), torch.cat(vs), torch.cat(seen, 1)
        s = torch.where(seen, q @ k.T * self.scale, -math.inf)
        z = torch.logsumexp(s, -1)
        p = (s - z[:, None]).exp()
        return p @ v, z / math.log(2.0), p.split(ranks, 1), p @ v.abs()

    def check(self, x):
        torch.cuda.synchronize()
        assert binding.device_status() == 0
        u = U[self.dtype]
        for b, n in enumerate(x["new"]):
            s = slice(x["start"][b], x["start"][b + 1])
            for h in range(self.H):
                if not n:
                    continue
                o, z, _, mass = self.expect(x, b, h)
                # P, the partials and the merged output are rounded once each; 2^-10 covers the 32-bit arithmetic
                tol = (2 * u + 2.0 ** -10) * mass + u * o.abs()
                err = (x["out"][s, h].double() - o).abs()
                assert bool((err <= tol).all()), (b, h, (err - tol).max().item())
                assert (x["out_lse"][s, h].double() - z).abs().max().item() <= 1e-4


def test_prompts_evictions_and_single_tokens():
    sv = Server()
    totals = torch.zeros((sv.N, sv.B, sv.Hkv, sv.cap), dtype=torch.float64, device=DEV)
    for new, pad in (([70, 1, 0], 2), ([130, 200, 33], 0), ([1, 0, 301], 1)):
        x = sv.batch(new, pad)
        sv.chunk(x)
        sv.check(x)
        assert bool((x["out"][sum(new):] == 0).all())
        for b, n in enumerate(new):
            for h in range(sv.H if n else 0):
                for r, p in enumerate(sv.expect(x, b, h)[2]):
                    totals[r, b, h // 4, :p.shape[1]] += p.sum(0)
    for b, l in enumerate(sv.lens):
        for r in range(sv.N):
            m = share(l, r, sv.N)
            got, want = sv.acc[r, b, :, :m].double(), totals[r, b, :, :m]
            assert bool(((got - want).abs() <= 1e-4 * want + 1e-5).all())
    before = {(r, b, h): sv.held(r, b, h) for r in range(sv.N) for b in range(sv.B) for h in range(sv.Hkv)}
    weight = sv.acc.clone()
    lens = list(sv.lens)
    kept = sv.evict(100, 24)
    torch.cuda.synchronize()
    for (r, b, h), (k, v, _) in before.items():
        k2, v2, i = sv.held(r, b, h)
        ids = kept[r, b, h, :len(i)].long()
        assert torch.equal(k2, k[ids]) and torch.equal(v2, v[ids]) and torch.equal(sv.acc[r, b, h, :len(i)],
                                                                                   weight[r, b, h][ids])
        late = [j for j in range(share(lens[b], r, sv.N)) if j * sv.N + r >= lens[b] - 24]
        assert set(late) <= set(ids.tolist())
        gone = [j for j in range(share(lens[b], r, sv.N)) if j not in set(ids.tolist())]
        older = [j for j in ids.tolist() if j not in late]
        if gone and older:
            assert weight[r, b, h][gone].max() <= weight[r, b, h][older].min()
    for _ in range(3):          # single tokens over what is left, their positions going on
        x = sv.batch([1, 1, 1])
        sv.decode(x)
        sv.check(x)
    x = sv.batch([5, 40, 1])    # and drafts
    sv.chunk(x)
    sv.check(x)


@pytest.mark.parametrize("D,page,dtype", [(64, 8, torch.float16), (256, 32, torch.bfloat16), (128, 2, torch.float16)])
def test_other_heads_and_pages(D, page, dtype):
    sv = Server(N=2, B=2, H=4, Hkv=2, D=D, page=page, max_len=500, dtype=dtype, seed=D)
    for new in ([90, 12], [40, 150], [1, 7]):
        x = sv.batch(new)
        sv.chunk(x)
        sv.check(x)
    sv.evict(60, 10)
    x = sv.batch([3, 20])
    sv.chunk(x)
    sv.check(x)


def test_a_captured_step_equals_the_eager_one():
    outs = []
    for captured in (False, True):
        sv = Server(seed=4)
        for new in ([70, 20, 0], [130, 1, 33]):
            x = sv.batch(new, 1)
            if not captured:
                sv.chunk(x)
                continue
            ws = torch.empty(binding.extend_workspace_bytes(sv.N, sv.B, x["T"], sv.H, sv.Hkv, sv.D, sv.max_len),
                             dtype=torch.uint8, device=DEV)
            acc, k, v = sv.acc.clone(), sv.k_pages.clone(), sv.v_pages.clone()
            sv.chunk(x, ws)                  # loads the kernels
            torch.cuda.synchronize()
            sv.acc.copy_(acc), sv.k_pages.copy_(k), sv.v_pages.copy_(v)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                sv.chunk(x, ws)
            for name in ("qn", "o", "lse", "out", "out_lse"):
                x[name].fill_(5.0)
            graph.replay()
        torch.cuda.synchronize()
        n = sum(x["new"])
        outs.append((x["out"][:n].clone(), x["out_lse"][:n].clone(), sv.acc.clone(), sv.k_pages.clone()))
    for a, b in zip(*outs):
        assert torch.equal(torch.nan_to_num(a.float(), nan=-7.0), torch.nan_to_num(b.float(), nan=-7.0))


def test_two_threads_on_their_own_streams():
    want, got, errors = {}, {}, []
    xs = {}
    for t in range(2):
        sv = Server(N=2 + t, H=8, Hkv=2 << t, seed=10 + t)
        xs[t] = (sv, [sv.batch([200, 30 + t, 5]) for _ in range(1)])
    torch.cuda.synchronize()

    def work(t, res):
        try:
            sv, batches = xs[t]
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    for x in batches:
                        sv.chunk(x)
            s.synchronize()
            res[t] = (batches[0]["out"].clone(), batches[0]["lse"].clone())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    for t in range(2):
        work(t, want)
    threads = [threading.Thread(target=work, args=(t, got)) for t in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors
    for t in range(2):
        assert torch.equal(want[t][0], got[t][0]) and torch.equal(want[t][1], got[t][1])
        xs[t][0].check(xs[t][1][0])


def test_host_tensors_and_long_lengths_are_refused():
    sv = Server(N=2, B=2, H=4, Hkv=2, max_len=100)
    x = sv.batch([20, 30])
    sv.append(x)
    args = [x["qn"], sv.k_pages, sv.v_pages, sv.table, x["qs"], x["sl"], sv.max_len, x["o"], x["lse"], sv.scale]
    for i in (0, 1, 2, 3, 4, 5, 7, 8):
        for host in (args[i].cpu(), args[i].cpu().pin_memory()):
            with pytest.raises(ValueError):
                binding.extend_attention_paged(*args[:i], host, *args[i + 1:])
    with pytest.raises(ValueError):
        binding.extend_attention_paged(*args[:6], (1 << 32) + sv.max_len, *args[7:])
    binding.extend_attention_paged(*args)


def test_a_recent_window_beyond_every_length_keeps_the_latest():
    sv = Server(N=2, B=2, H=4, Hkv=2, max_len=100)
    x = sv.batch([60, 90])
    sv.append(x)
    sv.acc.uniform_(0, 1, generator=sv.g)
    keep = torch.tensor([20, 31], dtype=torch.int32, device=DEV)
    outs = []
    for recent in (100, 1 << 40):
        kept = torch.full((2, 2, 2, 50), -1, dtype=torch.int32, device=DEV)
        out = torch.full((2, 2, 2, 50), math.nan, device=DEV)
        binding.cache_evict_paged(sv.k_pages, sv.v_pages, sv.table, x["sl"], 100, sv.acc, keep, 1 << 40, recent, sv.spare,
                                  kept, out)
        outs.append(kept)
    assert torch.equal(*outs)
    for b, (n, k) in enumerate(((60, 20), (90, 31))):
        for r in range(2):
            held, some = share(n, r, 2), share(k, r, 2)
            want = torch.arange(held - some, held, dtype=torch.int32, device=DEV)
            assert (outs[0][r, b, :, :some] == want).all() and (outs[0][r, b, :, some:] == -1).all()


STALL = r"""
import os, sys
sys.path[:0] = [sys.argv[1], os.path.join(sys.argv[1], "tests")]
import torch
from decode_context_attention_gb300 import binding
from test_chunk_serving_gpu import Server
for D in (64, 128):
    sv = Server(N=2, B=2, H=4, Hkv=2, D=D, max_len=300)
    x = sv.batch([40, 100])
    sv.append(x)
    args = (x["qn"], sv.k_pages, sv.v_pages, sv.table, x["qs"], x["sl"], sv.max_len, x["o"], x["lse"], sv.scale)
    wargs = (x["qn"], sv.k_pages, sv.table, x["qs"], x["sl"], sv.max_len, x["out_lse"], sv.acc, sv.scale)
    for call in (lambda: binding.extend_attention_paged(*args), lambda: binding.attention_weights_paged(*wargs)):
        os.environ["DCP_TEST_STALL_LOADS"] = "1"
        call()
        torch.cuda.synchronize()
        assert binding.device_status() == 7, "expected DCP_ERR_TIMEOUT"
        assert binding.device_status() == 0, "the status must clear once read"
        del os.environ["DCP_TEST_STALL_LOADS"]
        call()
        torch.cuda.synchronize()
        assert binding.device_status() == 0
    sv.acc.zero_()
    sv.chunk(x)
    sv.check(x)
print("timeouts reported, context usable")
"""


def test_waits_that_run_out_are_reported_and_leave_the_context_usable():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ)
    env.pop("DCP_TEST_STALL_LOADS", None)
    r = subprocess.run([sys.executable, "-c", STALL, root], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "timeouts reported, context usable" in r.stdout
