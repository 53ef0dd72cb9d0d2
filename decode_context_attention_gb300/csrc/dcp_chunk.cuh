// dcp_chunk.cuh -- device helpers of the chunk kernels (append, chunk
// attention, accumulated weights, eviction): a ragged batch's requests, the
// round-robin share of a rank, rows of the paged caches, and the split of a
// ragged batch's attention over the CTAs.
#pragma once

#include <math.h>

#include "dcp_chain.cuh"
#include "dcp_device.cuh"

namespace dcp {

// Rank r's share of the first n tokens of a request (sglang PR #33926 report,
// "关键源码片段", `get_dcp_lens`).
__device__ __forceinline__ int rank_share(int n, int r, int N) { return n <= 0 ? 0 : n / N + (r < n % N ? 1 : 0); }

struct Request {
    int start, n, L;  // first row, new tokens, tokens in all
};

// Whatever query_start and seq_lens hold, rows stay in [0, T) and lengths in
// [0, max_seq_len].
__device__ __forceinline__ Request load_request(const ChunkParams& p, int b) {
    const int s = min(max(__ldg(p.query_start + b), 0), p.T);
    const int e = min(max(__ldg(p.query_start + b + 1), s), p.T);
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len);
    return {s, e - s, L};
}

// A request as the plan of a batch that shares prefixes has it: the common part of a
// group (the rows of all its requests, tokens before them) or a request's own part
// (tokens from table entry `first` on, their number a multiple of N before it, so that
// the round-robin shares of what is left stay those of a request that begins there).
enum { kAlone = 0, kCommon = 1, kOwn = 2 };
struct Planned : Request {
    int b, first;  // row of the block table, first entry
    int kind;      // kAlone: no common part, nothing to join
    int common;    // kOwn: the index of its common part
};
template <class P>
struct RequestOf {
    using type = Request;
};
template <>
struct RequestOf<PrefixParams> {
    using type = Planned;
};
// (Plain loads: the kernel that reads the plan starts before the one that writes it ends, and what is read through
// the read-only path must not change while a kernel runs; such a load may also move over the wait.)
__device__ __forceinline__ Planned load_planned(const int4* at) {
    const int4 a = at[0], b = at[1];
    Planned q;
    q.start = a.x; q.n = a.y; q.L = a.z; q.b = a.w;
    q.first = b.x; q.kind = b.y; q.common = b.z;
    return q;
}
__device__ __forceinline__ Planned load_request(const PrefixParams& p, int v) {
    return load_planned(p.plan + 2 * (int64_t)v);
}
__device__ __forceinline__ bool is_causal(const ChunkParams& p, const Request&) { return p.causal != 0; }
__device__ __forceinline__ bool is_causal(const PrefixParams& p, const Planned& q) {
    return p.causal && q.kind != kCommon;
}

// Local tokens of rank r that new token j of the request sees.
template <class P, class R>
__device__ __forceinline__ int visible(const P& p, const R& q, int j, int r) {
    return rank_share(is_causal(p, q) ? q.L - q.n + j + 1 : q.L, r, p.N);
}

// Where the table entries of (rank, request b = q) begin.
__device__ __forceinline__ int64_t table_at(const ChunkParams& p, const Request&, int r, int b) {
    return (int64_t)r * p.bt_sn + (int64_t)b * p.bt_sb;
}
__device__ __forceinline__ int64_t table_at(const PrefixParams& p, const Planned& q, int r, int) {
    return (int64_t)r * p.bt_sn + (int64_t)q.b * p.bt_sb + q.first;
}
// Page of local token i from the entries at `at`, or -1 when they name none of the pool's.
__device__ __forceinline__ int page_in(const ChunkParams& p, int64_t at, int i) {
    const int pg = __ldg(p.bt + at + (i >> p.page_shift));
    return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
}

// Page of local token i, or -1 when the table names none of the pool's.
__device__ __forceinline__ int page_of(const ChunkParams& p, int r, int b, int i) {
    const int pg = __ldg(p.bt + (int64_t)r * p.bt_sn + (int64_t)b * p.bt_sb + (i >> p.page_shift));
    return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
}
__device__ __forceinline__ int64_t k_offset(const ChunkParams& p, int r, int pg, int i, int hkv) {
    return (int64_t)r * p.k_sn + (int64_t)pg * p.k_sp + (int64_t)(i & ((1 << p.page_shift) - 1)) * p.k_st +
           (int64_t)hkv * p.k_sh;
}
__device__ __forceinline__ int64_t v_offset(const ChunkParams& p, int r, int pg, int i, int hkv) {
    return (int64_t)r * p.v_sn + (int64_t)pg * p.v_sp + (int64_t)(i & ((1 << p.page_shift) - 1)) * p.v_st +
           (int64_t)hkv * p.v_sh;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by ex2.approx (at most 2 ulp off; 2^-inf = 0): the exponentials of a
// softmax, whose argument already carries a larger rounding error.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations an instruction, each rounded to nearest, on pairs held in one
// 64-bit register.
using Pair = unsigned long long;
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ void add2(Pair& a, Pair b) { asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b)); }

// sum over i < n of floor((a i + b) / m), for b >= 0, m > 0: whole multiples of m in a
// and b come out in closed form, and what is left counts the lattice points under a
// line, which read from the other axis is a sum of the same kind with m and a swapped
// (the classical reduction, as in Graham, Knuth, Patashnik, "Concrete Mathematics",
// chapter 3, and in the sum-of-floors routines of algorithm collections).  32-bit
// divisions where the terms fit.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    auto div = [](int64_t x, int64_t y) -> int64_t {
        return ((x | y) >> 32) ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
    };
    int64_t sum = 0;
    while (n > 0) {
        if (a >= m) {
            const int64_t k = div(a, m);
            sum += n * (n - 1) / 2 * k;
            a -= k * m;
        }
        if (b >= m) {
            const int64_t k = div(b, m);
            sum += n * k;
            b -= k * m;
        }
        const int64_t y = a * n + b;  // a and b below m <= 2^20, n below 2^31
        if (y < m) break;
        n = div(y, m);
        b = y - n * m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// ---------------------------------------------------------------------------
// The split of a ragged batch's attention.  An item is (request, rank, KV head,
// block of `tpi` new tokens); its work is the tiles of `tt` cached tokens its
// rows see, dearer when the item has more new tokens than `half` (it then fills
// both row blocks of a CTA), plus a fixed part.  The items' total is cut into `ctas` equal
// ranges: a range starts and ends inside items, so every CTA has the same work
// whatever the mix of long and short requests, and a single request with a
// long cache is split over all of them.  Items that are cut leave partial
// results, at most two per CTA, that a merge joins.
// ---------------------------------------------------------------------------
struct ChunkPos {
    int b, rh, qt, tile;  // request, rank * Hkv + KV head, block of new tokens, first tile; b = B at the end
};
__device__ __forceinline__ bool same_item(const ChunkPos& x, const ChunkPos& y) {
    return x.b == y.b && x.rh == y.rh && x.qt == y.qt;
}

// Tiles that block qt of the request sees on rank r.
template <class P, class R>
__device__ __forceinline__ int item_tiles(const P& p, const R& q, int r, int qt, int tpi, int tt) {
    const int last = min((qt + 1) * tpi, q.n) - 1;
    return (visible(p, q, last, r) + tt - 1) / tt;
}

// The first request from b on that has new tokens, or B.  Whole warps, the same b in all lanes.
__device__ __forceinline__ int next_request(const ChunkParams& p, int b) {
    while (b < p.B && load_request(p, b).n == 0) ++b;
    return b;
}
// In a plan all slim requests have none: they are passed 32 at a time.  (One by one they took 0.3 us each, in the chunk
// kernel and again in the join: a chunk of 300 in front of 255 single tokens 163 us, now 47; behind some millions the
// other warps' waits for the next part ran out.  The extend, which rarely meets one, is 1% slower with this.)
__device__ __forceinline__ int next_request(const PrefixParams& p, int b) {
    const int lane = threadIdx.x & 31;
    while (b < p.B) {
        const unsigned on = __ballot_sync(0xffffffffu, load_request(p, min(b + lane, p.B - 1)).n > 0);
        if (on) return b + __ffs(on) - 1;  // (lanes behind the last request see what its lane, before them, sees)
        b += 32;
    }
    return p.B;
}

// The first position of the item after `x`; as above.
template <class P>
__device__ __forceinline__ ChunkPos next_item(const P& p, const ChunkPos& x, int tpi) {
    ChunkPos y = x;
    y.tile = 0;
    if (++y.qt * tpi < load_request(p, y.b).n) return y;
    y.qt = 0;
    if (++y.rh < p.N * p.Hkv) return y;
    y.rh = 0;
    y.b = next_request(p, y.b + 1);
    return y;
}

constexpr int kPairTile = 4, kBlockTile = 3;  // work of a tile of two row blocks, and of one
constexpr int kItemCost = 13;                 // fixed part of an item's work (about 4.8 us against 1.5 us a pair's tile)
// Chosen on a mixed batch of 17 requests at D = 64: 145 us; with 4, 3, 9: 147, with 4, 3,
// 18: 160, with 2, 1, 5: 165.  At D = 128, where a tile costs more, 23 requests with 8
// heads a group take 413, with 18 386; 17 with a head a group 222 and 221; 5 requests
// 49.9, with 9 47.1 and with 18 51.4: no setting is best for all
constexpr int kMinPart = 4;   // a cut leaves at least this many tiles on both sides

// The work of one KV head of a (request, rank), by blocks of new tokens.
struct HeadWork {
    int nq;       // blocks
    int last;     // tiles of the last one
    int q0;       // blocks that see nothing because the request has more new tokens than tokens
    int wf, wl;   // weight of a tile: of a full block, of the last one
    int64_t a, b, m;
    __device__ int weight(int q) const { return q < nq - 1 ? wf : wl; }
};
template <class P>
__device__ inline HeadWork head_work(const P& p, int pair, int tpi, int half, int tt) {
    HeadWork w;
    const int r = pair % p.N;
    const auto q = load_request(p, pair / p.N);
    w.nq = (q.n + tpi - 1) / tpi;
    w.last = (rank_share(q.L, r, p.N) + tt - 1) / tt;  // its last row is the request's last token
    w.q0 = 0;
    w.wf = tpi > half ? kPairTile : kBlockTile;
    w.wl = q.n - (w.nq - 1) * tpi > half ? kPairTile : kBlockTile;
    w.m = (int64_t)p.N * tt;
    if (is_causal(p, q)) {
        // block qt's last row has x = L - n + (qt + 1) tpi tokens before or at it: rank_share(x) =
        // floor((x + N - 1 - r) / N), tiles = floor((x + m - 1 - r) / m), 0 below zero
        w.a = tpi;
        w.b = (int64_t)q.L - q.n + tpi + w.m - 1 - r;
        if (w.b < 0) {
            w.q0 = (int)((-w.b + tpi - 1) / tpi);
            w.b += (int64_t)w.q0 * tpi;
        }
    } else {
        w.a = 0;
        w.b = w.last * w.m;
    }
    return w;
}
// Work of the blocks before q.
__device__ inline int64_t work_before(const HeadWork& w, int q) {
    const int k = min(q, w.nq - 1) - w.q0;
    int64_t c = (int64_t)q * kItemCost;
    if (k > 0) c += w.wf * floor_sum(k, w.m, w.a, w.b);
    if (q >= w.nq && w.nq > 0) c += (int64_t)w.wl * w.last;
    return c;
}

// The start of range c of `ctas`.  upto[t] is the work up to and with the pairs of
// slot t (`per` (request, rank) pairs each, `slots` slots).  One warp, whose lanes
// try as many places of a search at once.
template <class P>
__device__ __forceinline__ ChunkPos range_start(const P& p, int tpi, int half, int tt, int ctas, int c,
                                                const int64_t* upto, int slots, int64_t per) {
    const unsigned all = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    ChunkPos x = {p.B, 0, 0, 0};
    const int64_t total = upto[slots - 1];
    const int64_t at = (int64_t)((double)total * c / ctas);  // exact below 2^53 / ctas, monotone above
    if (c >= ctas || at >= total) return x;
    // the last place of [lo, hi] for which before(place) <= at holds: it does for lo, and up to some place
    auto search = [&](int lo, int hi, auto before) {
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32;
            const int n = __popc(__ballot_sync(all, before(min(lo + (lane + 1) * step, hi))));
            const int next = n < 32 ? min(lo + (n + 1) * step, hi) - 1 : hi;
            lo = min(lo + n * step, hi);
            hi = max(next, lo);
        }
        return lo;
    };
    // the first slot whose pairs pass `at`
    const int slot = search(0, slots - 1, [&](int k) { return upto[k - 1] <= at; });
    int64_t rem = at - (slot ? upto[slot - 1] : 0);
    int64_t pair = slot * per;
    HeadWork w = head_work(p, (int)pair, tpi, half, tt);
    int64_t head = work_before(w, w.nq);
    while (rem >= head * p.Hkv) {  // `at` lies in one of this slot's pairs
        rem -= head * p.Hkv;
        w = head_work(p, (int)++pair, tpi, half, tt);
        head = work_before(w, w.nq);
    }
    const int b = (int)(pair / p.N), r = (int)(pair - (int64_t)b * p.N);
    const int hkv = (int)(rem / head);
    rem -= hkv * head;
    // the last block whose work starts at or before rem
    const int q0 = search(0, w.nq - 1, [&](int k) { return work_before(w, k) <= rem; });
    const int64_t begin = work_before(w, q0 + (lane & 1));  // of q0 and of the block after it
    const int weight = w.weight(q0);
    const int work = (int)(__shfl_sync(all, begin, 1) - __shfl_sync(all, begin, 0)) - kItemCost;
    const int off = (int)(rem - __shfl_sync(all, begin, 0));
    const int n = work / weight;
    x = {b, r * p.Hkv + hkv, q0, max(off - kItemCost, 0) / weight};
    // a cut near an end of its item, or into a short one, moves to the nearer end
    if (2 * off < work + kItemCost) {
        if (x.tile < kMinPart || n < 2 * kMinPart) x.tile = 0;
    } else if (n - x.tile < kMinPart || n < 2 * kMinPart) {
        x = next_item(p, x, tpi);
    }
    return x;
}

// Every CTA finds its own range: range[0] and range[1], with the starts of all
// ranges left in pos for the merge.  `scratch` holds THREADS + 32 numbers.  All
// threads of the CTA; ends with a barrier.
template <int THREADS, class P>
__device__ __forceinline__ void find_range(const P& p, int tpi, int half, int tt, ChunkPos* pos,
                                           int64_t* scratch, ChunkPos* range) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t npairs = (int64_t)p.B * p.N;
    const int64_t per = (npairs + THREADS - 1) / THREADS;
    int64_t sum = 0;
    for (int64_t i = tid * per; i < min((tid + 1) * per, npairs); ++i) {
        const HeadWork w = head_work(p, (int)i, tpi, half, tt);
        sum += work_before(w, w.nq) * p.Hkv;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) scratch[THREADS + warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += scratch[THREADS + w];
    scratch[tid] = sum;
    __syncthreads();
    if (warp < 2) {
        const int c = (int)blockIdx.x + warp;
        const ChunkPos x = range_start(p, tpi, half, tt, (int)gridDim.x, c, scratch, THREADS, per);
        if (lane == 0) {
            range[warp] = x;
            if (warp == 0 || c == (int)gridDim.x) pos[c] = x;
        }
    }
    __syncthreads();
}

// A CTA's part of an item.
template <class R>
struct ChunkSegOf {
    int b, r, hkv;
    int row0, nrows;     // first token row, rows (token, head) of the item
    int j0;              // first new token of the item within its request
    int t0, t1;          // tiles [t0, t1) of its ntiles
    int lim0, lim_last;  // tokens its first and its last row see: the tiles from lim0 / tt on are masked
    int slot;            // where a partial result goes, -1 when the part is the whole item
    int64_t table;       // where the request's table entries begin
    R q;
};
template <class P>
using ChunkSegFor = ChunkSegOf<typename RequestOf<P>::type>;
template <class P>
__device__ __forceinline__ ChunkSegFor<P> load_seg(const P& p, const ChunkPos& x, const ChunkPos& first,
                                                   const ChunkPos& end, int tpi, int tt) {
    ChunkSegFor<P> s;
    s.b = x.b;
    s.r = x.rh / p.Hkv;
    s.hkv = x.rh - s.r * p.Hkv;
    s.q = load_request(p, x.b);
    s.table = table_at(p, s.q, s.r, s.b);
    s.j0 = x.qt * tpi;
    const int tokens = min(tpi, s.q.n - s.j0);
    s.row0 = s.q.start + s.j0;
    s.nrows = tokens * p.gq;
    s.lim0 = visible(p, s.q, s.j0, s.r);
    s.lim_last = visible(p, s.q, s.j0 + tokens - 1, s.r);
    const int ntiles = (s.lim_last + tt - 1) / tt;
    s.t0 = x.tile;
    s.t1 = same_item(x, end) ? end.tile : ntiles;
    s.slot = s.t0 == 0 && s.t1 == ntiles ? -1 : 2 * (int)blockIdx.x + (same_item(x, first) ? 0 : 1);
    return s;
}

// Where the partials of cut items and the ranges lie in the workspace.
struct ChunkPartials {
    ChunkPos* pos;  // [ctas + 1]
    float* o;       // [2 * ctas][rows][D]
    float* lse;     // [2 * ctas][rows], base 2
};
size_t chunk_partials_bytes(int ctas, int rows, int D);
ChunkPartials chunk_partials_in(unsigned char* ws, int ctas, int rows, int D);
// Joins the cut items (rows of an item: tpi tokens x gq heads, at most `rows`); nothing
// to do, and no launch, when no item is long enough to be cut.
cudaError_t launch_chunk_merge(const ChunkParams& p, const ChunkPartials& ws, int tpi, int tt, int rows, int ctas,
                               int dtype, cudaStream_t stream);

// For a batch that shares prefixes: which own parts are slim, and what follows the chunk
// kernel (rows of an item: tpi tokens x gq heads, at most `rows`): slim parts, and the
// join of common and own parts.
// (`maps`: room for two tensor maps, which the finish reads on the host.)
void slim_limits(PrefixParams& p, int dtype, void* maps);
cudaError_t launch_prefix_finish(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                                 cudaStream_t stream);

// Where the row of a part goes in fp32 when it is not the whole result: the slot of a
// cut item, else the plan's row of a part that is joined; -1: the output itself.
__device__ __forceinline__ int64_t partial_row(const ChunkParams&, const Request&, int, int64_t, int) { return -1; }
__device__ __forceinline__ int64_t partial_row(const PrefixParams& p, const Planned& q, int r, int64_t t, int h) {
    if (q.kind == kAlone) return -1;
    return (((int64_t)(q.kind - 1) * p.N + r) * p.T + t) * p.H + h;
}
__device__ __forceinline__ float* partial_o(const ChunkParams&) { return nullptr; }
__device__ __forceinline__ float* partial_o(const PrefixParams& p) { return p.wo; }
__device__ __forceinline__ float* partial_lse(const ChunkParams&) { return nullptr; }
__device__ __forceinline__ float* partial_lse(const PrefixParams& p) { return p.wl; }

// Adds what the tokens set in `mask` (local tokens tile0 + bit, tokens whose V row
// holds NaN or infinities and was zeroed for the product) give to a row that
// sees them (i < lim): out[d] += p_i v_i[d] for the elements that are not
// finite.  `table`: where the request's entries begin.  lse2 is the row's base-2 log-sum-exp.  One thread, a rare path.
template <typename T, typename O>
__device__ __noinline__ void add_nonfinite(const ChunkParams& p, int r, int64_t table, int hkv, const T* q, int tile0,
                                           const unsigned* mask, int words, int lim, float lse2, O* out) {
    for (int w = 0; w < words; ++w) {
        for (unsigned m = mask[w]; m; m &= m - 1) {
            const int i = tile0 + 32 * w + __ffs(m) - 1;
            if (i >= lim) return;
            const int pg = page_in(p, table, i);
            if (pg < 0) continue;
            const T* k = reinterpret_cast<const T*>(p.k + k_offset(p, r, pg, i, hkv));
            const T* v = reinterpret_cast<const T*>(p.v + v_offset(p, r, pg, i, hkv));
            float s = 0.f;
            for (int d = 0; d < p.D; ++d) s = fmaf(to_f32(q[d]), to_f32(k[d]), s);
            const float pr = exp2f(s * p.sm_scale * kLog2e - lse2);
            for (int d = 0; d < p.D; ++d) {
                const float x = to_f32(v[d]);
                if (!isfinite(x)) out[d] = from_f32<O>(to_f32(out[d]) + pr * x);
            }
        }
    }
}

}  // namespace dcp
