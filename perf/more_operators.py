"""Shared prefixes and page bookkeeping of the round-robin paged caches, as measured work.

Three operators that a serving loop runs around its attention: pages and index
arrays of a step's new tokens built from the requests' lengths (`reserve`), the
attention of a batch whose requests share a long prefix (`prefix`), and the way of
pages back to the free lists (`release`).

Layouts: q [T, H, D]; pages [N, num_pages, page, Hkv, D]; block_table [N, B,
max_pages]; free_pages [N, capacity] with free_count [N], a stack for each rank.
Token g of a request lives on rank g % N as local token g // N.  Requests
group_start[g]..group_start[g+1] have their first prefix_lens[g] tokens in common,
and the whole pages of these are the first request's.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, dtype="bf16", N=4, B=64, H=32, Hkv=4, D=128, page=64, q=1, own_len=1024, prefix=0, groups=1,
          ragged=False, shape=1, pad=0, **more):
    c = dict(op=op, dtype=dtype, N=N, B=B, H=H, Hkv=Hkv, D=D, page=page, q=q, own_len=own_len, prefix=prefix,
             groups=groups, ragged=ragged, shape=shape, pad=pad)
    if name:
        c["name"] = name
    c.update(more)
    return c


def listed():
    return [
        # the bookkeeping of one decode step of 64 requests, each of which begins a page
        _case("reserve", "reserve_decode_B64", B=64, q=1, own_len=2049),
        # a prefill batch of eight 2048-token chunks behind a common system prompt
        _case("reserve", "reserve_chunk_T16384", B=8, q=2048, own_len=4096, prefix=2048),
        # thousands of small requests in 64 groups, single tokens and drafts, small pages
        _case("reserve", "reserve_ragged_B4096", N=8, B=4096, page=16, q=8, own_len=2000, prefix=1500, groups=64,
              ragged=True, shape=7, pad=33),
        # a batch of 64 ends, or is moved to the pages an eviction filled
        _case("release", "release_B64", B=64, q=1, own_len=8192, ended=1.0),
        # a fifth of thousands of requests ends, some are cut back to their prefix
        _case("release", "release_ragged_B4096", N=8, B=4096, page=16, q=8, own_len=2000, prefix=1500, groups=64,
              ragged=True, shape=9, ended=0.2),
        # a small batch behind a short system prompt: latency
        _case("prefix", "prefix_small_B8", N=1, B=8, own_len=200, prefix=1024),
        # a decode step of 64 requests behind one long document
        _case("prefix", "prefix_decode_B64", B=64, own_len=1024, prefix=32768),
        # a decode step of many requests behind a system prompt, the ordinary case
        _case("prefix", "prefix_decode_B256", B=256, own_len=700, prefix=2048, ragged=True, shape=4),
        # drafts of four tokens verified, two documents, large heads' groups
        _case("prefix", "prefix_verify_B48_Q4", N=2, B=48, H=64, Hkv=4, q=4, own_len=512, prefix=16384, groups=2),
        # chunks of prompts behind a common document: products bound it
        _case("prefix", "prefix_chunk_Q512", N=1, B=8, q=512, own_len=1024, prefix=16384),
        # several groups of odd sizes and lengths, loose requests, every query head its own keys
        _case("prefix", "prefix_groups_D64", dtype="f16", N=2, B=37, H=16, Hkv=16, D=64, page=16, q=5, own_len=777,
              prefix=5003, groups=5, ragged=True, shape=3, pad=5),
        # wide heads
        _case("prefix", "prefix_decode_D256", N=1, B=32, H=16, Hkv=2, D=256, own_len=512, prefix=8192),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("reserve", "release", "prefix", "prefix"))
    N = rng.choice((1, 2, 3, 4, 8))
    page = rng.choice((8, 16, 32, 64, 128))
    ragged, shape, dtype = rng.random() < 0.6, rng.randrange(1, 1 << 20), rng.choice(("bf16", "f16"))
    if op != "prefix":
        B, own_len, prefix = _logint(rng, 1, 4096), _logint(rng, 16, 16384), rng.choice((0, _logint(rng, 64, 16384)))
        most = (1 << 22) * page // (N * B) * N     # entries of the tables
        own_len, prefix = max(16, min(own_len, most // 2)), min(prefix, most // 2)
        q = max(1, min(_logint(rng, 1, 2048), own_len, 32768 // B))
        more = dict(ended=rng.choice((0.1, 0.5, 1.0))) if op == "release" else {}
        return _case(op, None, dtype, N, B, 32, 4, 128, page, q, own_len, prefix, rng.randrange(1, min(B, 64) + 1),
                     ragged, shape, rng.choice((0, 0, 3)), **more)
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8))
    H = Hkv * rng.choice((1, 2, 4, 8, 12, 16))
    B, q = _logint(rng, 1, 200), rng.choice((1, 1, _logint(rng, 1, 300)))
    own_len = max(q, _logint(rng, 16, 2000))
    own_len = max(16, min(own_len, (1 << 25) // (B * Hkv * D)))
    q = max(1, min(q, own_len, 4096 // B))
    prefix = max(64, min(_logint(rng, 64, 32768), (1 << 29) // (B * q * H)))
    return _case(op, None, dtype, N, B, H, Hkv, D, page, q, own_len, prefix, rng.randrange(1, min(B, 6) + 1), ragged,
                 shape, rng.choice((0, 0, 3)), causal=rng.random() < 0.9)


def _plan(case):
    """New tokens and total lengths of every request, the groups' borders and prefixes.  A ragged batch has groups of
    one, requests behind the last group, a request that only holds its group's prefix, single tokens and chunks."""
    r = random.Random(case["shape"])
    B, G, q, p, o = (case[k] for k in ("B", "groups", "q", "prefix", "own_len"))
    if not p:
        G = 0
    if case["ragged"]:
        loose = r.randrange(B // 4 + 1)
        G = min(G, B - loose)
        cuts = sorted(r.sample(range(1, B - loose), G - 1)) if G > 1 else []
        border = [0] * (G > 0) + cuts + [B - loose] * (G > 0)
        plen = [r.randint(1, p) for _ in range(G)]
        if G:
            plen[r.randrange(G)] = p
    else:
        border = [B * g // G for g in range(G + 1)] if G else []
        plen = [p] * G
    of = [-1] * B
    for g in range(G):
        of[border[g]:border[g + 1]] = [g] * (border[g + 1] - border[g])
    qs, ls = [], []
    for b in range(B):
        base = _shared(case, plen[of[b]]) if of[b] >= 0 else 0
        if not case["ragged"]:
            qs.append(q)
            ls.append(max(base + o, plen[of[b]] + q if of[b] >= 0 else 0))
            continue
        n = r.choice((0, 1)) if r.random() < 0.3 else r.randint(1, q)
        low = plen[of[b]] if of[b] >= 0 else 0
        qs.append(n)
        ls.append(n + r.randint(low, max(low, base + o - n)))
    return qs, ls, border, plen, of


def _shared(case, p):
    """Tokens in the whole pages, on every rank, of a prefix of p."""
    unit = case["N"] * case["page"]
    return p // unit * unit


def _share(n, r, N):
    return n // N + (1 if r < n % N else 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    N, B, ps = case["N"], case["B"], case["page"]
    qs, ls, border, plen, of = _plan(case)
    start = [0]
    for n in qs:
        start.append(start[-1] + n)
    n_new, max_len = start[-1], max(ls)
    T = n_new + case["pad"]
    mp = -(-(-(-max_len // N)) // ps)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case=case, n_new=n_new, T=T, max_len=max_len, query_start=ints(start), seq_lens=ints(ls),
             group_start=ints(border) if border else None, prefix_lens=ints(plen) if border else None,
             plan=(qs, ls, border, plen, of), shared=[_shared(case, plen[i]) if i >= 0 else 0 for i in of])
    lens, news = ints(ls).long(), ints(qs).long()
    group = torch.tensor(of, device=dev)
    first = torch.tensor([border[i] if i >= 0 else b for b, i in enumerate(of)], device=dev)
    whole = torch.tensor(s["shared"], device=dev) // (N * ps)
    rank, b = torch.arange(N, device=dev)[:, None], torch.arange(B, device=dev)
    need = -(-(lens // N + (rank < lens % N)) // ps)                       # entries a request has on each rank
    held = need if case["op"] != "reserve" else -(-((lens - news) // N + (rank < (lens - news) % N)) // ps)
    skip = torch.where(first == b, 0, whole)
    # pages of the pool are handed out in no order; a member's common pages are the first request's
    own_pages = (held - skip).clamp(min=0)
    total = int((need - skip).clamp(min=0).sum(1).max())
    pages = total + 7
    perm = torch.stack([torch.randperm(pages, generator=g, device=dev) for _ in range(N)])
    j = torch.arange(mp, device=dev)
    at = own_pages.cumsum(1) - own_pages
    at = (at - skip)[..., None] + j
    mine = (j >= skip[..., None]) & (j < held[..., None])
    table = torch.where(mine, perm.gather(1, at.clamp(0, pages - 1).flatten(1)).view_as(at), -1)
    common = (j < whole[:, None]) & (first != b)[:, None] & (j < held[..., None])
    s["block_table"] = torch.where(common, table[:, first], table).int()
    used = own_pages.sum(1)
    s["num_pages"] = pages
    if case["op"] in ("reserve", "release"):
        free = torch.stack([torch.cat([perm[r, int(used[r]):], perm.new_full((int(used[r]),), -1)]) for r in range(N)])
        s["free_pages"], s["free_count"] = free.int(), (pages - used).int()
        s["free_out"] = torch.zeros_like(s["free_count"])
    if case["op"] == "reserve":
        s["cached_lens"], s["new_lens"] = (lens - news).int(), news.int()
        s["query_start"], s["seq_lens"] = torch.zeros_like(s["query_start"]), torch.zeros_like(s["seq_lens"])
        s["missing"] = ints([0] * N)
        s["positions"], s["requests"] = ints([0] * T), ints([0] * T)
        s["slots"] = torch.zeros(T, dtype=torch.int64, device=dev)
    elif case["op"] == "release":
        r = random.Random(case["shape"] + seed)
        keep = [(0 if r.random() < 0.7 else s["shared"][i] + r.randrange(64)) if r.random() < case["ended"] else -1
                for i in range(B)]
        # a request that holds its group's prefix stays
        for i in range(B):
            if of[i] >= 0 and border[of[i]] == i and border[of[i] + 1] > i + 1:
                keep[i] = -1
        s["keep_lens"], s["lens_out"] = ints(keep), ints([0] * B)
    else:
        H, Hkv, D, dt = case["H"], case["Hkv"], case["D"], DTYPES[case["dtype"]]
        s["sm_scale"] = D ** -0.5
        normal = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=dt)  # noqa: E731
        s["k_pages"], s["v_pages"] = normal(N, pages, ps, Hkv, D), normal(N, pages, ps, Hkv, D)
        # normalised queries; some heads look sharply, some broadly
        temp = torch.empty(H, 1, device=dev).uniform_(0.5, 2.5, generator=g)
        s["q"] = (normal(T, H, D) * temp).to(dt)
        s["o"] = torch.zeros(N, T, H, D, dtype=dt, device=dev)
        s["lse"] = torch.zeros(N, T, H, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        from decode_context_attention_gb300 import binding
        c = s["case"]
        if op == "reserve":
            binding.page_reserve(s["cached_lens"], s["new_lens"], s["max_len"], s["T"], s["num_pages"], c["page"],
                                 s["block_table"], s["free_pages"], s["free_count"], s["free_out"], s["missing"],
                                 s["query_start"], s["seq_lens"], positions=s["positions"], slots=s["slots"],
                                 requests=s["requests"], group_start=s["group_start"], prefix_lens=s["prefix_lens"])
        elif op == "release":
            binding.page_release(s["seq_lens"], s["keep_lens"], s["max_len"], s["num_pages"], c["page"],
                                 s["block_table"], s["free_pages"], s["free_count"], s["free_out"],
                                 lens_out=s["lens_out"], group_start=s["group_start"], prefix_lens=s["prefix_lens"])
        else:
            binding.prefix_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["query_start"],
                                           s["seq_lens"], s["max_len"], s["group_start"], s["prefix_lens"], s["o"],
                                           s["lse"], s["sm_scale"], causal=c.get("causal", True))
    else:
        {"reserve": _reserve, "release": _release, "prefix": _prefix}[op](s)
    if op == "reserve":
        names = ("block_table", "free_out", "missing", "query_start", "seq_lens", "positions", "slots", "requests")
    elif op == "release":
        names = ("free_pages", "free_out", "lens_out")
    else:
        names = ("o", "lse")
    return {k: s[k] for k in names}


def _groups(s, B, N, ps):
    """The first request of every request's group (itself outside of groups), and the entries it has from it."""
    dev = s["block_table"].device
    b = torch.arange(B, device=dev)
    if s["group_start"] is None:
        return b, torch.zeros_like(b)
    gs, pl = s["group_start"].long(), s["prefix_lens"].long()
    g = torch.searchsorted(gs[1:], b, right=True)
    inside = (b >= gs[0]) & (b < gs[-1])
    g = g.clamp(max=pl.shape[0] - 1)
    first = torch.where(inside, gs[g], b)
    return first, torch.where(first != b, pl[g] // (N * ps), 0)


def _entries(n, N, ps):
    rank = torch.arange(N, device=n.device)[:, None]
    return (n // N + (rank < n % N) + ps - 1) // ps


def _reserve(s):
    c, table = s["case"], s["block_table"]
    N, B, ps, dev = c["N"], c["B"], c["page"], table.device
    mp = table.shape[2]
    cached = s["cached_lens"].long()
    n = torch.minimum(s["new_lens"].long(), s["max_len"] - cached).clamp(min=0)
    s["query_start"][1:] = n.cumsum(0).clamp(max=s["T"]).int()
    s["query_start"][0] = 0
    n = (s["query_start"][1:] - s["query_start"][:-1]).long()
    L = cached + n
    s["seq_lens"].copy_(L)
    first, common = _groups(s, B, N, ps)
    have = torch.maximum(_entries(cached, N, ps), common)
    want = _entries(L, N, ps)
    count = (want - have).clamp(min=0)
    left = s["free_count"].long()
    j = torch.arange(mp, device=dev)
    k = (count.cumsum(1) - count - have)[..., None] + j
    at = left[:, None, None] - 1 - k
    page = s["free_pages"].gather(1, at.clamp(0, s["free_pages"].shape[1] - 1).flatten(1)).view_as(at)
    page = torch.where(at >= 0, page, -1)
    table.copy_(torch.where((j >= have[..., None]) & (j < want[..., None]), page, table))
    table.copy_(torch.where(j < common[:, None], table[:, first], table))
    s["free_out"].copy_((left - count.sum(1)).clamp(min=0))
    s["missing"].copy_((count.sum(1) - left).clamp(min=0))
    t = torch.arange(int(s["n_new"]), device=dev)
    qs = s["query_start"].long()
    b = torch.searchsorted(qs[1:], t, right=True)
    g = cached[b] + t - qs[b]
    r, i = g % N, g // N
    page = table[r, b, i // ps].long()
    slot = torch.where((page >= 0) & (page < s["num_pages"]), (r * s["num_pages"] + page) * ps + i % ps, -1)
    s["positions"][: t.shape[0]] = g.int()
    s["slots"][: t.shape[0]] = slot
    s["requests"][: t.shape[0]] = b.int()


def _release(s):
    c, table, free = s["case"], s["block_table"], s["free_pages"]
    N, B, ps, dev = c["N"], c["B"], c["page"], table.device
    L, keep = s["seq_lens"].long(), s["keep_lens"].long()
    keep = torch.where(keep < 0, L, torch.minimum(keep, L))
    _, common = _groups(s, B, N, ps)
    low, high = torch.maximum(_entries(keep, N, ps), common), _entries(L, N, ps)
    j = torch.arange(table.shape[2], device=dev)
    gone = (j >= low[..., None]) & (j < high[..., None]) & (table >= 0) & (table < s["num_pages"])
    gone = gone.flatten(1)
    at = s["free_count"].long()[:, None] + gone.long().cumsum(1) - 1
    rank = torch.arange(N, device=dev)[:, None].expand_as(at)
    fits = gone & (at < free.shape[1])
    free[rank[fits], at[fits]] = table.flatten(1)[fits]
    s["free_out"].copy_((s["free_count"].long() + gone.sum(1)).clamp(max=free.shape[1]))
    s["lens_out"].copy_(keep)


def _rows(s, pages, table, lo, hi):
    """Local tokens [lo, hi) of every rank from rows [N, ..., max_pages] of the table, in 32 bits: [N, ..., tokens,
    Hkv, D]."""
    ps = s["case"]["page"]
    i = torch.arange(lo, hi, device=pages.device)
    p = table[..., (i // ps).clamp(max=table.shape[-1] - 1)].long().clamp(0, s["num_pages"] - 1)
    r = torch.arange(pages.shape[0], device=pages.device).view(-1, *([1] * (p.dim() - 1)))
    return pages[r, p, i % ps].float()


def _prefix(s):
    c, dev = s["case"], s["q"].device
    N, B, H, Hkv, D = (c[k] for k in ("N", "B", "H", "Hkv", "D"))
    qs, ls, border, plen, of = s["plan"]
    start = [sum(qs[:b]) for b in range(B + 1)]
    causal, n_new = c.get("causal", True), s["n_new"]
    q = s["q"][:n_new].float().view(n_new, Hkv, H // Hkv, D)
    m = torch.full((N, n_new, Hkv, H // Hkv), -math.inf, device=dev)
    l = torch.zeros_like(m)
    o = torch.zeros(N, n_new, Hkv, H // Hkv, D, device=dev)

    def attend(at, x, v, seen, form):
        """Adds scores x with values v to the rows `at` of the running softmax."""
        x = x if seen is None else x.masked_fill(~seen, -math.inf)
        new = torch.maximum(m[:, at], x.amax(-1))
        base = torch.where(new == -math.inf, torch.zeros_like(new), new)
        p = (x - base[..., None]).exp_()
        old = (m[:, at] - base).exp()
        o[:, at] = o[:, at] * old[..., None] + torch.einsum(form, p, v)
        l[:, at] = l[:, at] * old + p.sum(-1)
        m[:, at] = new

    # the common whole pages, once for all the rows of a group
    for g in range(len(plen)):
        lo, hi = start[border[g]], start[border[g + 1]]
        end = _shared(c, plen[g]) // N
        if lo < hi and end:
            row = s["block_table"][:, border[g]]
            k, v = _rows(s, s["k_pages"], row, 0, end), _rows(s, s["v_pages"], row, 0, end)
            x = torch.einsum("thgd,nihd->nthgi", q[lo:hi], k) * s["sm_scale"]
            attend(slice(lo, hi), x, v, None, "nthgi,nihd->nthgd")
            del x
    # every request's own tokens, a few requests at a time
    some = max(1, (1 << 28) // max(1, H * max(qs) * max(c["own_len"], 64)))
    shared = torch.tensor(s["shared"], device=dev)
    busy = [b for b in range(B) if qs[b]]
    for b0 in range(0, len(busy), some):
        bs = busy[b0: b0 + some]
        bt = torch.tensor(bs, device=dev)
        Q = max(qs[b] for b in bs)
        width = max(-(-(ls[b] - s["shared"][b]) // N) for b in bs)
        if not width:
            continue
        i = (shared[bt] // N)[:, None] + torch.arange(width, device=dev)
        entry = (i // c["page"]).clamp(max=s["block_table"].shape[2] - 1)
        p = s["block_table"][:, bt].gather(2, entry.expand(N, -1, -1)).long()
        p = p.clamp(0, s["num_pages"] - 1)
        rank = torch.arange(N, device=dev)[:, None, None]
        k, v = s["k_pages"][rank, p, i % c["page"]].float(), s["v_pages"][rank, p, i % c["page"]].float()
        n = (s["query_start"][1:] - s["query_start"][:-1]).long()[bt]
        j = torch.arange(Q, device=dev)
        real = j < n[:, None]
        rows = (s["query_start"].long()[bt][:, None] + j).clamp(max=n_new - 1)
        L = s["seq_lens"].long()[bt]
        last = (L - n)[:, None] + j if causal else (L - 1)[:, None].expand(-1, Q)
        seen = (i * N + rank)[:, :, None, :] <= last[:, :, None]
        x = torch.einsum("bqhgd,nbihd->nbqhgi", q[rows], k) * s["sm_scale"]
        x = x.masked_fill_(~seen[:, :, :, None, None], -math.inf)
        new = torch.maximum(m[:, rows], x.amax(-1))
        base = torch.where(new == -math.inf, torch.zeros_like(new), new)
        x = x.sub_(base[..., None]).exp_()
        old = (m[:, rows] - base).exp()
        to = rows[real]
        o[:, to] = (o[:, rows] * old[..., None] + torch.einsum("nbqhgi,nbihd->nbqhgd", x, v))[:, real]
        l[:, to] = (l[:, rows] * old + x.sum(-1))[:, real]
        m[:, to] = new[:, real]
        del x
    o = torch.where(l[..., None] > 0, o / l[..., None], torch.zeros_like(o))
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    s["o"][:, :n_new] = o.flatten(2, 3).to(s["o"].dtype)
    s["lse"][:, :n_new] = (base + l.log()).flatten(2, 3)


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------

def work(case):
    N, B, H, Hkv, D, ps = (case[k] for k in ("N", "B", "H", "Hkv", "D", "page"))
    qs, ls, border, plen, of = _plan(case)
    shared = [_shared(case, plen[g]) if g >= 0 else 0 for g in of]
    T = sum(qs)
    entries = lambda n: sum(-(-_share(n, r, N) // ps) for r in range(N))  # noqa: E731
    if case["op"] == "reserve":
        new = sum(max(0, entries(L) - max(entries(L - n), s // ps)) for n, L, s in zip(qs, ls, shared))
        common = sum(s // ps for b, s in enumerate(shared) if s and border[of[b]] != b)
        return {"bytes": 16 * B + 8 * new + 4 * common + 16 * T, "flops": 0}
    if case["op"] == "release":
        gone = case["ended"] * sum(entries(L) - s // ps for L, s in zip(ls, shared))
        return {"bytes": 12 * B + 8 * int(gone), "flops": 0}
    pairs = tokens = 0
    for n, L, s in zip(qs, ls, shared):
        pairs += n * (L - n) + n * (n + 1) // 2 if case.get("causal", True) else n * L
        tokens += L - s if n else 0
    for g in range(len(plen)):
        tokens += _shared(case, plen[g]) if any(qs[border[g]:border[g + 1]]) else 0
    return {"bytes": 2 * T * H * D + 4 * tokens * Hkv * D + N * T * H * (2 * D + 4), "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# the definitions, one request at a time (attention in 64 bits)
# ---------------------------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    qs, ls, border, plen, of = s["plan"]
    N, B, ps = case["N"], case["B"], case["page"]
    table = s["block_table"].cpu().numpy()
    if case["op"] == "reserve":
        free, count = s["free_pages"].tolist(), s["free_count"].tolist()
        missing, starts, pos, slots, req = [0] * N, [0], [], [], []
        for b in range(B):
            starts.append(starts[-1] + qs[b])
            first = border[of[b]] if of[b] >= 0 else b
            for r in range(N):
                have = -(-_share(ls[b] - qs[b], r, N) // ps)
                if first != b:
                    have = max(have, s["shared"][b] // N // ps)
                for j in range(have, -(-_share(ls[b], r, N) // ps)):
                    if count[r]:
                        count[r] -= 1
                        table[r, b, j] = free[r][count[r]]
                    else:
                        table[r, b, j] = -1
                        missing[r] += 1
            if first != b:
                w = s["shared"][b] // N // ps
                table[:, b, :w] = table[:, first, :w]
            for g in range(ls[b] - qs[b], ls[b]):
                page = int(table[g % N, b, g // N // ps])
                pos.append(g)
                req.append(b)
                slots.append(((g % N) * s["num_pages"] + page) * ps + g // N % ps if page >= 0 else -1)
        pad = [0] * case["pad"]
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"block_table": ints(table), "free_out": ints(count), "missing": ints(missing),
                "query_start": ints(starts), "seq_lens": ints(ls), "positions": ints(pos + pad),
                "slots": torch.tensor(slots + pad, dtype=torch.int64, device="cuda"), "requests": ints(req + pad)}
    if case["op"] == "release":
        free, count, keep, lens = s["free_pages"].cpu().numpy(), s["free_count"].tolist(), s["keep_lens"].tolist(), []
        for b in range(B):
            lens.append(ls[b] if keep[b] < 0 else min(keep[b], ls[b]))
            inner = of[b] >= 0 and border[of[b]] != b
            for r in range(N):
                low = -(-_share(lens[b], r, N) // ps)
                if inner:
                    low = max(low, s["shared"][b] // N // ps)
                gone = table[r, b, low: max(low, -(-_share(ls[b], r, N) // ps))]
                free[r, count[r]: count[r] + len(gone)] = gone
                count[r] += len(gone)
        return {"free_pages": torch.tensor(free, device="cuda"),
                "free_out": torch.tensor(count, dtype=torch.int32, device="cuda"),
                "lens_out": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    o, lse = s["o"].double(), s["lse"].double()
    G, at = case["H"] // case["Hkv"], 0
    for b, (n, L) in enumerate(zip(qs, ls)):
        rows = slice(at, at + n)
        at += n
        if not n:
            continue
        last = L - n + torch.arange(n, device="cuda") if case.get("causal", True) else torch.full((n,), L, device="cuda")
        for r in range(N):
            m = _share(L, r, N)
            if not m:
                o[r, rows], lse[r, rows] = 0.0, -math.inf
                continue
            i = torch.arange(m, device="cuda")
            page = s["block_table"][r, b].long()[i // ps]
            k, v = (x[r, page, i % ps].double().repeat_interleave(G, 1).transpose(0, 1)
                    for x in (s["k_pages"], s["v_pages"]))                           # [H, m, D]
            x = torch.bmm(s["q"][rows].double().transpose(0, 1), k.transpose(1, 2)) * s["sm_scale"]
            seen = (i * N + r)[None, :] <= last[:, None]
            x = torch.where(seen, x, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.where(seen, (x - z[..., None]).exp(), 0.0)
            lse[r, rows] = z.T
            o[r, rows] = torch.bmm(p, v).transpose(0, 1)
    return {"o": o, "lse": lse}
