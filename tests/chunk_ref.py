"""Ragged batches over round-robin paged caches, and the chunk operators'
definitions in 64 bits (one request, rank and head at a time), with the error
bounds their arithmetic allows."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}      # half a step of a subnormal
DEV = "cuda"


def share(n, r, N):
    return 0 if n <= 0 else n // N + (1 if r < n % N else 0)


class Batch:
    """Requests of `lens` = [(new tokens, tokens in all), ...] over pools whose pages are shuffled; everything a
    request does not own holds NaN."""

    def __init__(self, lens, N=2, H=8, Hkv=2, D=128, page=16, dtype=torch.bfloat16, pad=0, seed=0, max_len=None,
                 strided=False, qscale=1.0):
        self.lens, self.N, self.H, self.Hkv, self.D, self.page, self.dtype = lens, N, H, Hkv, D, page, dtype
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.g = g
        B = len(lens)
        self.B, self.T = B, sum(n for n, _ in lens) + pad
        self.max_len = max_len if max_len is not None else max([l for _, l in lens] + [1])
        self.cap = -(-self.max_len // N)
        mp = max(1, -(-self.cap // page))
        start = [0]
        for n, _ in lens:
            start.append(start[-1] + n)
        self.start = start
        self.query_start = torch.tensor(start, dtype=torch.int32, device=DEV)
        self.seq_lens = torch.tensor([l for _, l in lens], dtype=torch.int32, device=DEV)
        pages = B * mp + 3
        self.num_pages = pages
        self.block_table = torch.full((N, B, mp), 2 ** 30, dtype=torch.int32, device=DEV)
        # [.., Hkv, 2, D] interleaved when strided: K and V side by side, other strides than a dense pool's
        if strided:
            both = torch.full((N, pages, page, Hkv, 2, D), float("nan"), dtype=dtype, device=DEV)
            self.k_pages, self.v_pages = both[..., 0, :], both[..., 1, :]
        else:
            self.k_pages = torch.full((N, pages, page, Hkv, D), float("nan"), dtype=dtype, device=DEV)
            self.v_pages = torch.full((N, pages, page, Hkv, D), float("nan"), dtype=dtype, device=DEV)
        self.k = [torch.randn((l, Hkv, D), generator=g, device=DEV).to(dtype) for _, l in lens]
        self.v = [torch.randn((l, Hkv, D), generator=g, device=DEV).to(dtype) for _, l in lens]
        for r in range(N):
            perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
            for b, (_, l) in enumerate(lens):
                own = -(-share(l, r, N) // page)
                self.block_table[r, b, :own] = perm[b * mp: b * mp + own]
        self.fill()
        if strided:
            wide = (torch.randn((self.T, H + 3, D + 8), generator=g, device=DEV) * qscale).to(dtype)
            self.q = wide[:, 1:H + 1, :D]
        else:
            self.q = (torch.randn((self.T, H, D), generator=g, device=DEV) * qscale).to(dtype)
        self.scale = D ** -0.5

    def slot(self, b, r, i):
        """(page, slot) of local tokens i (a tensor) of request b on rank r."""
        return self.block_table[r, b].long()[i // self.page], i % self.page

    def fill(self):
        for b, (_, l) in enumerate(self.lens):
            for r in range(self.N):
                i = torch.arange(share(l, r, self.N), device=DEV)
                if len(i):
                    pg, sl = self.slot(b, r, i)
                    self.k_pages[r, pg, sl] = self.k[b][i * self.N + r]
                    self.v_pages[r, pg, sl] = self.v[b][i * self.N + r]

    def rows(self, b):
        return slice(self.start[b], self.start[b + 1])

    def limits(self, b, r, causal=True):
        """Visible local tokens of every new token of request b on rank r."""
        n, l = self.lens[b]
        g = [l - n + j + 1 if causal else l for j in range(n)]
        return torch.tensor([share(x, r, self.N) for x in g], device=DEV)

    def scores(self, b, r, h):
        """Scores [n, m] in 64 bits, and a bound on the kernels' error in them: sums of D exact products in 32 bits
        (each partial sum off by at most 2^-23 of the sum of magnitudes), times the scale."""
        m = share(self.lens[b][1], r, self.N)
        i = torch.arange(m, device=DEV)
        k = self.k[b][i * self.N + r, h // (self.H // self.Hkv)].double()
        q = self.q[self.rows(b), h].double()
        s = q @ k.T * self.scale
        err = (q.abs() @ k.nan_to_num().abs().T) * self.scale * (self.D / 8 + 4) * 2.0 ** -24
        return s, err


def attention(bt, causal=True):
    """o [N,T,H,D], lse [N,T,H] (base e) in 64 bits and their error bounds; rows of no request stay 0."""
    N, T, H, D = bt.N, bt.T, bt.H, bt.D
    o = torch.zeros((N, T, H, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((N, T, H), dtype=torch.float64, device=DEV)
    o_tol, lse_tol = torch.zeros_like(o), torch.zeros_like(lse)
    u, tiny = U[bt.dtype], TINY[bt.dtype]
    for b in range(bt.B):
        at = bt.rows(b)
        if not bt.lens[b][0]:
            continue
        for r in range(N):
            lim = bt.limits(b, r, causal)
            m = share(bt.lens[b][1], r, N)
            if m == 0:
                lse[r, at] = -math.inf
                continue
            i = torch.arange(m, device=DEV)
            seen = i[None] < lim[:, None]
            for h in range(H):
                s, err = bt.scores(b, r, h)
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
                err = torch.where(seen, err, torch.zeros_like(err)).amax(-1)
                z = torch.logsumexp(s, -1)
                p = torch.where(seen, (s - z[:, None]).exp(), torch.zeros_like(s))
                v = bt.v[b][i * N + r, h // (H // bt.Hkv)].double()
                want = torch.zeros((len(lim), D), dtype=torch.float64, device=DEV)
                if v.isfinite().all():
                    want = p @ v
                else:      # only what a row sees reaches it
                    for j in range(len(lim)):
                        want[j] = p[j, :lim[j]] @ v[:lim[j]]
                o[r, at, h], lse[r, at, h] = want, z
                mass = p @ v.nan_to_num(0.0, 0.0, 0.0).abs()
                # a weight: its score's error, ex2.approx and the sums (2^-18 in all), and P's rounding; the output's
                o_tol[r, at, h] = (u + 3 * err[:, None] + 2.0 ** -18) * mass + u * want.nan_to_num(0.0, 0.0, 0.0).abs() + tiny
                lse_tol[r, at, h] = 2 * err + 2.0 ** -20 + 2.0 ** -22 * z.nan_to_num(0.0, 0.0, 0.0).abs()
    return o, lse, o_tol, lse_tol


def weights(bt, lse, acc):
    """The accumulated weights in 64 bits, and their error bound; lse [T,H] base e."""
    out = acc.double().clone()
    tol = torch.zeros_like(out)
    G = bt.H // bt.Hkv
    for b, (n, l) in enumerate(bt.lens):
        if not n:
            continue
        for r in range(bt.N):
            m = share(l, r, bt.N)
            if not m:
                continue
            i = torch.arange(m, device=DEV)
            seen = i[None] < bt.limits(b, r)[:, None]
            old = i * bt.N + r < l - n
            for kh in range(bt.Hkv):
                new = torch.where(old, out[r, b, kh, :m], torch.zeros_like(out[r, b, kh, :m]))
                t = new.abs() * 2.0 ** -23
                for h in range(kh * G, (kh + 1) * G):
                    s, err = bt.scores(b, r, h)
                    z = lse[bt.rows(b), h].double()
                    on = seen & z.isfinite()[:, None]
                    w = torch.where(on, (s - z[:, None]).exp(), torch.zeros_like(s))
                    # the exponent: its score, the log-sum-exp in base 2 and their difference; the exponential; the sums
                    rel = 2 * err + 2.0 ** -22 * (s.abs() + z.nan_to_num(0.0, 0.0, 0.0).abs()[:, None]) + 2.0 ** -20
                    rel = rel + n * G * 2.0 ** -24
                    new = new + w.sum(0)
                    t = t + torch.where(on, w * rel, torch.zeros_like(w)).sum(0)
                out[r, b, kh, :m] = new
                tol[r, b, kh, :m] = t + 2.0 ** -24 * new.abs()
    return out, tol


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape
    fin = want.isfinite()
    assert torch.equal(fin, got.isfinite()), f"{what}: finite at other places"
    assert torch.equal(want.isnan(), got.isnan()), f"{what}: NaN at other places"
    assert torch.equal(got[~fin & ~want.isnan()], want[~fin & ~want.isnan()]), f"{what}: infinities"
    d = torch.where(fin, (got - want).abs() - tol, torch.zeros_like(want))
    worst = d.max().item() if d.numel() else 0.0
    assert worst <= 0, f"{what}: {int((d > 0).sum())} of {d.numel()} elements off by up to {worst:.3e} beyond the bound"
