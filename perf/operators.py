"""The chunk-serving operators over round-robin paged caches, as measured work.

Four operators around one cache: the query/key norm and rotation with the append
of K and V (`append`), the attention of a chunk of new tokens (`extend`), the
accumulated attention weights (`weights`) and the eviction by them (`evict`).

Layouts: q [T, H, D]; pages [N, num_pages, page, Hkv, D]; block_table [N, B,
max_pages]; request b owns the rows query_start[b]..query_start[b+1] of q, its
last new tokens, out of seq_lens[b] in all.  Token g of a request lives on rank
g % N as local token g // N.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, name=None, dtype="bf16", N=4, B=1, H=32, Hkv=4, D=128, page=64, q=1, l=4096, ragged=False, shape=1,
          pad=0, **more):
    c = dict(op=op, dtype=dtype, N=N, B=B, H=H, Hkv=Hkv, D=D, page=page, q=q, l=l, ragged=ragged, shape=shape, pad=pad)
    if name:
        c["name"] = name
    c.update(more)
    return c


def listed():
    return [
        # one decode step's new tokens of 64 requests: a launch, and little else
        _case("append", "append_decode_B64", B=64, q=1, l=2048, rot=128, interleaved=False),
        # a prefill batch of eight 2048-token chunks
        _case("append", "append_chunk_T16384", B=8, q=2048, l=4096, rot=128, interleaved=False),
        # ragged chunks, small heads of which half is rotated in neighbouring pairs, rows behind the last sequence
        _case("append", "append_ragged_D64", dtype="f16", N=2, B=13, H=16, Hkv=16, D=64, page=16, q=1021, l=2500,
              ragged=True, shape=7, pad=11, rot=32, interleaved=True),
        # drafts of four tokens verified for 32 requests with long caches: the cache is read, and that is the cost
        _case("extend", "extend_verify_B32_Q4", B=32, q=4, l=16384, ragged=False, causal=True),
        # one prompt chunk against its own tokens and 6k earlier ones
        _case("extend", "extend_chunk_Q2048", N=1, B=2, q=2048, l=8192, causal=True),
        # the last chunk of a long prompt: products bound it
        _case("extend", "extend_long_Q4096", N=4, B=1, q=4096, l=32768, causal=True),
        # single tokens and chunks in one batch, odd lengths, every query head its own keys
        _case("extend", "extend_mixed_D64", dtype="f16", N=2, B=17, H=16, Hkv=16, D=64, page=16, q=517, l=4999,
              ragged=True, shape=3, pad=5, causal=True),
        # the weights of a decode step: reads the keys once
        _case("weights", "weights_decode_B64", B=64, q=1, l=8192),
        # the weights of a prompt chunk: half of an attention's products
        _case("weights", "weights_chunk_Q2048", N=2, B=1, q=2048, l=16384),
        # odd lengths, 12 query heads to a key head
        _case("weights", "weights_ragged_G12", N=8, B=9, H=96, Hkv=8, page=32, q=67, l=6001, ragged=True, shape=5, pad=3),
        # 32 requests cut to half their tokens
        _case("evict", "evict_B32_half", B=32, l=8192, keep=4096, recent=256),
        # one long prompt compressed once
        _case("evict", "evict_long_131072", N=2, B=1, Hkv=8, l=131072, keep=8192, recent=512),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("append", "extend", "weights", "evict"))
    D = rng.choice((64, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 8))
    gq = rng.choice((1, 2, 4, 8, 12, 16))
    H = Hkv * gq
    N = rng.choice((1, 2, 3, 4, 8))
    more = {}
    if op == "append":
        B, q = _logint(rng, 1, 64), _logint(rng, 1, 1024)
        q = max(1, min(q, 16384 // B, (1 << 26) // (B * H * D)))
        l = q + rng.randrange(0, 1000)
        half = rng.random() < 0.3
        more = dict(rot=D // 2 if half else D, interleaved=rng.random() < 0.3)
    elif op == "evict":
        B, q = _logint(rng, 1, 32), 0
        l = _logint(rng, 64, 65536)
        l = max(64, min(l, (1 << 25) // (B * Hkv * D)))
        keep = max(1, int(l * rng.uniform(0.05, 1.0)))
        more = dict(keep=keep, recent=rng.choice((0, 1, 64, max(1, keep // 4))))
    else:
        B, l = _logint(rng, 1, 48), _logint(rng, 32, 20000)
        l = max(32, min(l, (1 << 25) // (B * Hkv * D)))
        q = min(_logint(rng, 1, 2048), l)
        q = max(1, min(q, (1 << 30) // (B * H * l)))
        if op == "extend":
            more = dict(causal=rng.random() < 0.8)
    return _case(op, None, rng.choice(("bf16", "f16")), N, B, H, Hkv, D, rng.choice((8, 16, 32, 64, 128)), q, l,
                 rng.random() < 0.6, rng.randrange(1, 1 << 20), rng.choice((0, 0, 3)), **more)


def _lens(case):
    """New tokens and total lengths of every request: a ragged batch holds single tokens, an empty request now and
    then, and one request of the largest size."""
    r = random.Random(case["shape"])
    B, q, l = case["B"], case["q"], case["l"]
    if not case["ragged"]:
        return [q] * B, [l] * B
    qs, ls = [], []
    for _ in range(B):
        qb = 0 if q == 0 else (r.choice((0, 1)) if r.random() < 0.3 else r.randint(1, q))
        qs.append(qb)
        ls.append(qb + r.randint(0, l - qb))
    b = r.randrange(B)
    qs[b], ls[b] = q, l
    return qs, ls


def _share(n, r, N):
    return n // N + (1 if r < n % N else 0)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    N, B, H, Hkv, D, ps = (case[k] for k in ("N", "B", "H", "Hkv", "D", "page"))
    qs, ls = _lens(case)
    start = [0]
    for n in qs:
        start.append(start[-1] + n)
    n_new = start[-1]
    T = n_new + case["pad"]
    cap = max(1, -(-case["l"] // N))          # local tokens a rank may hold of one request
    mp = -(-cap // ps)
    s = dict(case=case, n_new=n_new, max_len=case["l"], q_max=max(1, case["q"]), cap=cap,
             query_start=torch.tensor(start, dtype=torch.int32, device=dev),
             seq_lens=torch.tensor(ls, dtype=torch.int32, device=dev), sm_scale=D ** -0.5)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=dt)

    # every request's pages are scattered over the pool; an evicting call also has pages to move into
    keep_cap = -(-case["keep"] // N) if case["op"] == "evict" else 0
    kp = -(-keep_cap // ps)
    pages = B * (mp + kp) + 3
    perm = torch.stack([torch.randperm(pages, generator=g, device=dev) for _ in range(N)]).to(torch.int32)
    s["block_table"] = perm[:, : B * mp].reshape(N, B, mp).contiguous()
    s["k_pages"], s["v_pages"] = normal(N, pages, ps, Hkv, D), normal(N, pages, ps, Hkv, D)
    if case["op"] == "append":
        # raw projections, in one buffer as a fused projection leaves them
        qkv = normal(T, H + 2 * Hkv, D) * 3
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dt)
        rot, P = case["rot"], case["l"] + 64
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        ang = torch.arange(P, dtype=torch.float64, device=dev)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float()
        s["positions"] = torch.tensor([ls[b] - qs[b] + j for b in range(B) for j in range(qs[b])] + [0] * case["pad"],
                                      dtype=torch.int32, device=dev)
        s["q_out"] = torch.zeros(T, H, D, dtype=dt, device=dev)
    elif case["op"] in ("extend", "weights"):
        # normalised queries; some heads look sharply, some broadly
        temp = torch.empty(H, 1, device=dev).uniform_(0.5, 2.5, generator=g)
        s["q"] = (normal(T, H, D) * temp).to(dt)
        if case["op"] == "extend":
            s["o"] = torch.zeros(N, T, H, D, dtype=dt, device=dev)
            s["lse"] = torch.zeros(N, T, H, device=dev)
        else:
            # the merge's log-sum-exp of random scores of variance temp^2 over the visible tokens, about
            seen = torch.tensor([ls[b] - qs[b] + j + 1 for b in range(B) for j in range(qs[b])] + [1] * case["pad"],
                                dtype=torch.float32, device=dev)
            s["lse"] = (seen.log()[:, None] + 0.5 * temp[None, :, 0] ** 2
                        + 0.1 * torch.randn(T, H, generator=g, device=dev)).contiguous()
            s["acc"] = torch.rand(N, B, Hkv, cap, generator=g, device=dev) * 4
    else:
        s["acc"] = torch.empty(N, B, Hkv, cap, device=dev).exponential_(1.0, generator=g)
        s["acc"] = (s["acc"] * 64).round() / 64       # ties, as counts of few queries have them
        s["keep_lens"] = torch.full((B,), case["keep"], dtype=torch.int32, device=dev)
        s["dst_table"] = perm[:, B * mp: B * (mp + kp)].reshape(N, B, kp).contiguous()
        s["kept"] = torch.full((N, B, Hkv, keep_cap), -1, dtype=torch.int32, device=dev)
        s["acc_out"] = torch.zeros(N, B, Hkv, keep_cap, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        from decode_context_attention_gb300 import binding
        c = s["case"]
        if op == "append":
            binding.qk_norm_rope_append(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS, s["cos_sin"],
                                        s["positions"], s["k_pages"], s["v_pages"], s["block_table"],
                                        s["query_start"], s["seq_lens"], s["max_len"], s["q_out"],
                                        interleaved=c["interleaved"])
        elif op == "extend":
            binding.extend_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["query_start"],
                                           s["seq_lens"], s["max_len"], s["o"], s["lse"], s["sm_scale"],
                                           causal=c["causal"])
        elif op == "weights":
            binding.attention_weights_paged(s["q"], s["k_pages"], s["block_table"], s["query_start"], s["seq_lens"],
                                            s["max_len"], s["lse"], s["acc"], s["sm_scale"])
        else:
            binding.cache_evict_paged(s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], s["max_len"],
                                      s["acc"], s["keep_lens"], c["keep"], c["recent"], s["dst_table"], s["kept"],
                                      s["acc_out"])
    else:
        {"append": _append, "extend": _extend, "weights": _weights, "evict": _evict}[op](s)
    if op == "append":
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "extend":
        return {"o": s["o"], "lse": s["lse"]}
    if op == "weights":
        return {"acc": s["acc"]}
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "kept": s["kept"], "acc": s["acc_out"]}


def _owners(s):
    """Request, index among its new tokens and global index of every new token."""
    t = torch.arange(s["n_new"], device=s["q"].device)
    qs, L = s["query_start"].long(), s["seq_lens"].long()
    b = torch.searchsorted(qs[1:], t, right=True)
    j = t - qs[b]
    return b, j, L[b] - (qs[b + 1] - qs[b]) + j


def _rotate(x, cos, sin, rot, interleaved):
    y, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., : rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _append(s):
    c, n = s["case"], s["n_new"]
    N, ps, rot = c["N"], c["page"], c["rot"]
    cs = s["cos_sin"][s["positions"][:n].long()][:, None]
    cos, sin = cs[..., : rot // 2], cs[..., rot // 2:]

    def norm(x, w):
        x = x[:n].float()
        return _rotate(x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float(), cos, sin, rot, c["interleaved"])

    s["q_out"][:n] = norm(s["q"], s["q_weight"]).to(s["q_out"].dtype)
    b, _, g = _owners(s)
    r, i = g % N, g // N
    page = s["block_table"][r, b, i // ps].long()
    s["k_pages"][r, page, i % ps] = norm(s["k"], s["k_weight"]).to(s["k_pages"].dtype)
    s["v_pages"][r, page, i % ps] = s["v"][:n]


def _cache(s, pages):
    """The caches of every rank and request as [N, B, Hkv, tokens, D] in 32 bits."""
    c = s["case"]
    r = torch.arange(c["N"], device=pages.device)[:, None, None]
    x = pages[r, s["block_table"].long()].flatten(2, 3)[:, :, : s["cap"]]
    return x.permute(0, 1, 3, 2, 4).float()


def _scores(s):
    """Scores [N, B, Hkv, G, Q, tokens] of the new tokens, and which of them are visible [N, B, 1, 1, Q, tokens]."""
    c = s["case"]
    N, B, H, Hkv, D = (c[k] for k in ("N", "B", "H", "Hkv", "D"))
    dev, Q = s["q"].device, s["q_max"]
    qs, L = s["query_start"].long(), s["seq_lens"].long()
    rows = (qs[:B, None] + torch.arange(Q, device=dev)).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[rows].view(B, Q, Hkv, H // Hkv, D).permute(0, 2, 3, 1, 4).reshape(1, B, Hkv, -1, D)
    sc = torch.matmul(q, _cache(s, s["k_pages"]).transpose(-1, -2)) * s["sm_scale"]
    sc = sc.view(N, B, Hkv, H // Hkv, Q, s["cap"])
    where = torch.arange(s["cap"], device=dev)[None, None, None, :] * N + torch.arange(N, device=dev)[:, None, None, None]
    old = (L - (qs[1:] - qs[:-1]))[None, :, None, None]
    last = old + torch.arange(Q, device=dev)[None, None, :, None] if c.get("causal", True) else L[None, :, None, None]
    seen = (where <= last) & (where < L[None, :, None, None])
    return sc, seen[:, :, None, None], where, old


def _extend(s):
    c, n = s["case"], s["n_new"]
    sc, seen, _, _ = _scores(s)
    sc = sc.masked_fill_(~seen, -math.inf)
    m = sc.amax(-1, keepdim=True)
    base = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(base).exp_()
    l = p.sum(-1, keepdim=True)
    N, B, Hkv, G, Q, _ = sc.shape
    o = torch.matmul(p.flatten(3, 4), _cache(s, s["v_pages"])).view(N, B, Hkv, G, Q, c["D"])
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (base + l.log())[..., 0]
    b, j, _ = _owners(s)
    s["o"][:, :n] = o.permute(0, 1, 4, 2, 3, 5).flatten(3, 4)[:, b, j].to(s["o"].dtype)
    s["lse"][:, :n] = lse.permute(0, 1, 4, 2, 3).flatten(3, 4)[:, b, j]


def _weights(s):
    c = s["case"]
    sc, seen, where, old = _scores(s)
    N, B, Hkv, G, Q, _ = sc.shape
    dev = sc.device
    qs, L = s["query_start"].long(), s["seq_lens"].long()
    rows = (qs[:B, None] + torch.arange(Q, device=dev)).clamp(max=s["q"].shape[0] - 1)
    lse = s["lse"][rows].view(B, Q, Hkv, G).permute(0, 2, 3, 1)[None, ..., None]
    real = (torch.arange(Q, device=dev) < (qs[1:] - qs[:-1])[:, None])[None, :, None, None, :, None]
    w = sc.sub_(lse).exp_().masked_fill_(~(seen & real & lse.isfinite()), 0.0).sum((3, 4))
    where, L = where[:, :, 0][:, :, None], L[None, :, None, None]
    acc = torch.where(where < old, s["acc"], torch.zeros_like(w)) + w
    s["acc"].copy_(torch.where(where < L, acc, s["acc"]))


def _evict(s):
    c = s["case"]
    N, ps, cap = c["N"], c["page"], s["cap"]
    acc, dev = s["acc"], s["acc"].device
    L, keep = s["seq_lens"].long(), s["keep_lens"].long()
    rank = torch.arange(N, device=dev)
    i = torch.arange(cap, device=dev)
    share = lambda n: (n[None, :] // N + (rank[:, None] < n[None, :] % N))[..., None, None]  # noqa: E731
    where = (i[None, None, None, :] * N + rank[:, None, None, None]).expand(N, c["B"], 1, cap)
    recent = where >= (L - c["recent"])[None, :, None, None]
    # classes: the recent window (latest first), the rest by weight (larger first), what is not there
    kind = torch.where(where >= L[None, :, None, None], 2, torch.where(recent, 0, 1)).expand_as(acc)
    value = torch.where(recent, i.float(), acc.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf))
    by_value = value.sort(dim=-1, descending=True, stable=True).indices
    order = by_value.gather(-1, kind.gather(-1, by_value).sort(dim=-1, stable=True).indices)
    k = share(torch.minimum(L, keep))
    kc = s["kept"].shape[-1]
    first = torch.arange(kc, device=dev)
    if kc > cap:
        order = torch.cat([order, order[..., :1].expand(*order.shape[:-1], kc - cap)], -1)
    real = (first < k).expand(*s["kept"].shape)
    src = torch.where(real, order[..., :kc], cap).sort(-1).values
    s["kept"].copy_(torch.where(real, src.int(), s["kept"]))
    src = src.clamp(max=cap - 1)
    s["acc_out"].copy_(torch.where(real, acc.gather(-1, src), s["acc_out"]))
    r, b, h = (torch.arange(n, device=dev).view(v) for n, v in
               ((N, (-1, 1, 1, 1)), (c["B"], (1, -1, 1, 1)), (c["Hkv"], (1, 1, -1, 1))))
    at = (r, s["block_table"][r, b, src // ps].long(), src % ps, h)
    to = (r, s["dst_table"][r, b, (first // ps)[None, None, None]].long(), (first % ps)[None, None, None], h)
    for pages in (s["k_pages"], s["v_pages"]):
        pages[to] = torch.where(real[..., None], pages[at], pages[to])


# ---------------------------------------------------------------------------
# what a pass has to move and compute
# ---------------------------------------------------------------------------

def work(case):
    N, B, H, Hkv, D = (case[k] for k in ("N", "B", "H", "Hkv", "D"))
    qs, ls = _lens(case)
    T, pairs = sum(qs), 0
    for q, l in zip(qs, ls):
        pairs += q * l if not case.get("causal", True) else q * (l - q) + q * (q + 1) // 2
    held = sum(l for q, l in zip(qs, ls) if q)      # tokens of requests that ask for anything
    if case["op"] == "append":
        return {"bytes": T * (4 * (H + 2 * Hkv) * D + 4 * case["rot"] + 4), "flops": T * (H + Hkv) * D * 7}
    if case["op"] == "extend":
        return {"bytes": 2 * T * H * D + 4 * held * Hkv * D + N * T * H * (2 * D + 4), "flops": 4 * D * H * pairs}
    if case["op"] == "weights":
        return {"bytes": T * H * (2 * D + 4) + 2 * held * Hkv * D + 8 * held * Hkv, "flops": 2 * D * H * pairs}
    kept = sum(min(l, case["keep"]) for l in ls)
    return {"bytes": Hkv * (4 * sum(ls) + kept * (8 * D + 8)), "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one request at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    qs, ls = _lens(case)
    N, H, Hkv, D, ps = (case[k] for k in ("N", "H", "Hkv", "D", "page"))
    G = H // Hkv
    starts = [sum(qs[:b]) for b in range(len(qs))]
    table = s["block_table"].tolist()
    if case["op"] == "append":
        rot, n = case["rot"], s["n_new"]
        d = torch.arange(rot, device="cuda")
        # element d of a rotated head is x[d] cos - x[partner] sin (first of its pair) or x[d] cos + x[partner] sin
        if case["interleaved"]:
            partner, angle, sign = d ^ 1, d // 2, (d % 2) * 2 - 1
        else:
            partner, angle, sign = (d + rot // 2) % rot, d % (rot // 2), (d >= rot // 2) * 2 - 1
        cs = s["cos_sin"].double()[s["positions"][:n].long()]
        cos, sin = cs[:, angle][:, None], (cs[:, rot // 2 + angle] * sign)[:, None]

        def turned(x, w):
            x = x[:n].double()
            x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()
            y = x.clone()
            y[..., :rot] = x[..., :rot] * cos + x[..., partner] * sin
            return y

        q = s["q_out"].double()
        q[:n] = turned(s["q"], s["q_weight"])
        k, kp, vp = turned(s["k"], s["k_weight"]), s["k_pages"].double(), s["v_pages"].double()
        at = [(g % N, table[g % N][b][g // N // ps], g // N % ps)
              for b in range(len(qs)) for g in range(ls[b] - qs[b], ls[b])]
        at = torch.tensor(at, device="cuda").unbind(-1)
        kp[at], vp[at] = k, s["v"][:n].double()
        return {"q": q, "k_pages": kp, "v_pages": vp}
    if case["op"] in ("extend", "weights"):
        o = s["o"].double() if "o" in s else None
        out = s["lse"].double() if "o" in s else s["acc"].double()
        for b, (n, L) in enumerate(zip(qs, ls)):
            if not n:
                continue
            at = slice(starts[b], starts[b] + n)
            g = L - n + torch.arange(n, device="cuda")
            for r in range(N):
                m = _share(L, r, N)
                if not m:
                    if o is not None:
                        o[r, at], out[r, at] = 0.0, -math.inf
                    continue
                i = torch.arange(m, device="cuda")
                page = s["block_table"][r, b].long()[i // ps]
                seen = (i * N + r)[None, :] <= (g if case.get("causal", True) else torch.full_like(g, L))[:, None]
                for h in range(H):
                    k = s["k_pages"][r, page, i % ps, h // G].double()
                    x = s["q"][at, h].double() @ k.T * s["sm_scale"]
                    if o is None:
                        w = torch.where(seen, (x - s["lse"][at, h].double()[:, None]).exp(), 0.0).sum(0)
                        if h % G == 0:
                            out[r, b, h // G, :m] *= i * N + r < L - n
                        out[r, b, h // G, :m] += w
                    else:
                        x = torch.where(seen, x, -math.inf)
                        lse = torch.logsumexp(x, -1)
                        out[r, at, h] = lse
                        p = torch.where(seen, (x - lse[:, None]).exp(), 0.0)
                        o[r, at, h] = p @ s["v_pages"][r, page, i % ps, h // G].double()
        return {"acc": out} if o is None else {"o": o, "lse": out}
    acc, kept, acc_out = s["acc"].cpu(), s["kept"], s["acc_out"].double()
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    k0, v0 = s["k_pages"], s["v_pages"]
    for b, L in enumerate(ls):
        for r in range(N):
            m, want = _share(L, r, N), _share(min(L, case["keep"]), r, N)
            for h in range(Hkv):
                a = acc[r, b, h, :m].tolist()
                late = [i for i in range(m) if i * N + r >= L - case["recent"]]
                pick = late[len(late) - min(want, len(late)):]
                rest = sorted((i for i in range(m - len(late))), key=lambda i: (-a[i], i))[: want - len(pick)]
                pick = sorted(rest + pick)
                if not pick:
                    continue
                p = torch.tensor(pick, device="cuda")
                kept[r, b, h, :want] = p.int()
                acc_out[r, b, h, :want] = s["acc"][r, b, h, p].double()
                to = torch.arange(want, device="cuda")
                src, dst = s["block_table"][r, b].long()[p // ps], s["dst_table"][r, b].long()[to // ps]
                kp[r, dst, to % ps, h] = k0[r, src, p % ps, h].double()
                vp[r, dst, to % ps, h] = v0[r, src, p % ps, h].double()
    return {"k_pages": kp, "v_pages": vp, "kept": kept, "acc": acc_out}
