// dcp_prefix_finish.cu -- the last step of the attention of a batch that shares
// prefixes: requests' own parts of few rows and tokens, and the join of every
// request's common and own parts.
//
// Joining parts over disjoint tokens with outputs o_i and log-sum-exps z_i:
//     z = log2 sum_i 2^z_i,  o = sum_i 2^(z_i - z) o_i.
//
// An own part of a decode step is a few rows (new tokens x heads of a group) over some
// hundred tokens: 100 to 300 KB of keys and values and hardly any arithmetic, which has to
// stream.  One to four warps take one (request, rank, KV head), 16 rows a warp, over every
// (second, fourth) tile of 16 tokens.  TMA fills a ring of tiles in shared memory, a box a
// page, so that a warp has two or more tiles under way and spends no instructions on them;
// ldmatrix and mma.sync (m16n8k16) take them from there.  (The same from global memory
// into the operands' registers, without shared memory: 60 us instead of 37 for 64 single
// tokens over 1024 own ones on 4 ranks; a warp waited for every tile, and spent twice the
// instructions on addresses and on pairing up values.)
// One pass, an online softmax with the reference maximum moved when it is passed by 2^8,
// as in the tensor-core kernel.  The kernel's code has to fit the instruction cache, as each
// CTA runs through it once: with a join of 110 KB of code 64 single tokens took 169 us in
// all, with one of 25 KB 127.
// Measured (bf16, 32 query heads over 4, D = 128, after the chunk kernel): 64 single tokens
// over 1024 own ones on 4 ranks 36 us, 156 MB, 4.3 TB/s; the loop itself runs at 7 TB/s, the
// rest is a launch, a chain of look-ups (plan, page, first tile: 4 us) and the join (5 us).
#include <cuda.h>
#include <stdlib.h>

#include <type_traits>

#include "dcp_chunk.cuh"
#include "dcp_mma.cuh"
#include "dcp_sm100.cuh"

namespace dcp {

using namespace sm100;

namespace {

__device__ int g_finish_status;  // first bounded wait that ran out (0 if none)

constexpr unsigned kAll = 0xffffffffu;
constexpr int kFinishThreads = 128;
constexpr int kMaxRanges = 512;  // CTAs of the kernel before

// A row's weights are 2^(s - m + kBias): fp16's smallest normal is 2^-14, and a largest
// weight of up to 2^15 keeps those of a long tail (dcp_chunk_attention_tc.cu).
constexpr float kGrow = 8.f;
template <typename T>
constexpr float kBias = std::is_same<T, __half>::value ? 7.f : 0.f;

constexpr int kTileTokens = 16;
constexpr int kMaxStages = 6;
template <int D>
struct Slim {
    static constexpr int WD = D == 256 ? 2 : 1;    // warps that share a tile's columns
    static constexpr int DW = D / WD;              // columns of a warp
    static constexpr int kBox = kTileTokens * 128;  // 64 columns of a tile, 128-byte swizzled
    static constexpr int kTile = 2 * (D / 64) * kBox;  // keys, then values
    // bytes of the ring for each warp that shares it.  With CTAs to spare three are on an SM, with two tiles a
    // warp (256 requests behind 2048 tokens 80 us; with three tiles and two CTAs 86); where two on each SM are
    // all there are, larger ones keep a third off an SM that is free first (64 behind 32768: 86, otherwise 90).
    static constexpr int kRingMany = D == 256 ? 24 * 1024 : 16 * 1024, kRingFew = D == 64 ? 16 * 1024 : 24 * 1024;
    static_assert(16 * D * 4 / WD <= kRingMany, "outputs lie where the ring was");
    static_assert(WD * kRingMany % kTile == 0 && WD * kRingFew % kTile == 0, "whole tiles");
};
struct SlimBars {
    uint64_t full[4][kMaxStages], empty[4][kMaxStages];  // by ring
    int abort;
};

// Where the parts of a common item lie: slots of the chunk kernel's partials, or (n = -1) the plan's rows.
struct Parts {
    int n;
    unsigned short slot[kMaxRanges + 1];
};

// The parts of the item, by one warp: the range that holds its first tile by two rounds of 32 at once.
__device__ __noinline__ void find_parts(const ChunkPos* pos, int ctas, const ChunkPos& item, Parts* parts) {
    const int lane = threadIdx.x & 31;
    auto begun = [&](const ChunkPos& x) {
        return x.b != item.b ? x.b < item.b : x.rh != item.rh ? x.rh < item.rh : x.qt != item.qt ? x.qt < item.qt : x.tile == 0;
    };
    const int step = (ctas + 32) / 32;  // of ctas + 1 places; at most 16
    const int n = __popc(__ballot_sync(kAll, lane * step <= ctas && begun(pos[min(lane * step, ctas)])));
    int base = max(n - 1, 0) * step;
    ChunkPos x = pos[min(base + lane, ctas)];
    const int m = __popc(__ballot_sync(kAll, lane < step && base + lane <= ctas && begun(x)));  // c = base + m - 1
    unsigned same = __ballot_sync(kAll, base + lane <= ctas && same_item(x, item));
    if (n == 0 || m == 0 || !(same >> m & 1)) {  // no range begins inside the item
        if (lane == 0) parts->n = -1;
        return;
    }
    if (lane == 0) parts->slot[0] = (unsigned short)(2 * (base + m - 1) + (same >> (m - 1) & 1 ? 0 : 1));
    int count = 1;
    for (int skip = m;; skip = 0) {
        // a range that lies empty inside the item left nothing
        int next_tile = __shfl_down_sync(kAll, x.tile, 1);
        bool next_same = lane < 31 && (same >> (lane + 1) & 1);
        if (lane == 31 && base + 32 <= ctas) {
            const ChunkPos y = pos[base + 32];
            next_tile = y.tile;
            next_same = same_item(y, item);
        }
        const bool in = lane >= skip && base + lane < ctas && (same >> lane & 1);
        const unsigned on = __ballot_sync(kAll, in && !(next_same && next_tile == x.tile));
        if (on >> lane & 1) parts->slot[count + __popc(on & ((1u << lane) - 1u))] =
                (unsigned short)(2 * (base + lane));
        count += __popc(on);
        if (!(same >> 31) || base + 32 >= ctas) break;
        base += 32;
        x = pos[min(base + lane, ctas)];
        same = __ballot_sync(kAll, base + lane <= ctas && same_item(x, item));
    }
    if (lane == 0) parts->n = count;
}

template <typename P>
__device__ __forceinline__ P* shfl_ptr(P* p, int lane) {
    return reinterpret_cast<P*>(__shfl_sync(kAll, (unsigned long long)p, lane));
}
// 1 / x within 1 ulp.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ const float4 g_zero_row[64] = {};  // of a part that is not there

// What a lane knows of its row of those that its warp joins: where the result goes (NULL:
// it is none), and how many parts it has.
struct JoinRow {
    unsigned char* out;
    float* lse;
    int parts;
};
// A part's outputs times its weight, the base-2 logarithm of their unit, and its weight: 1 beside a log-sum-exp.
struct Part {
    const float* o;
    float z, weight;
};
// The join of a warp's `count` rows (a power of two up to 8): lane k has row k & (count - 1)
// and the parts k / count, k / count + 32 / count, ... of it, part(n) saying where they lie
// (in global or shared memory).  32 parts at a time: their weights are the lanes', one each,
// so that what is left for all lanes is a load and an FMA an element.
template <typename T, int D, class Get>
__device__ __forceinline__ void join_rows(const PrefixParams& p, int count, const JoinRow& row, Get part) {
    constexpr int NV = (D + 127) / 128, kBatch = 16 / NV;  // parts in flight
    const int lane = threadIdx.x & 31;
    const bool wide = 4 * lane < D;  // (half a warp holds a row of 64)
    const float* const zeros = reinterpret_cast<const float*>(g_zero_row);
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 a[8][NV];  // of the rows 0 to 7; with fewer, shares of them
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int v = 0; v < NV; ++v) a[e][v] = none;
    float m = -INFINITY, sum = 0.f;
    const int clog = count == 8 ? 3 : count >> 1, step = 32 >> clog;
    const int most = (int)__reduce_max_sync(kAll, (unsigned)row.parts);
#pragma unroll 1
    for (int i = 0; i < most; i += step) {
        Part x = {zeros, -INFINITY, 0.f};
        const bool there = i + (lane >> clog) < row.parts;
        if (there) x = part(i + (lane >> clog));
        // all the rows' lines on their way at once (of shared memory: no operation)
        if (there)
#pragma unroll
            for (int l = 0; l < D; l += 32) asm volatile("prefetch.L2 [%0];" ::"l"(x.o + l));
        float top = x.z;
#pragma unroll 1
        for (int d = count; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, d));
        top = fmaxf(top, m);
        // the reference becomes finite or infinite with the parts, and a NaN part's weight NaN: as the formula has it
        const float base = top == -INFINITY ? 0.f : top;
        const float old = exp2_fast(m - base), w = exp2_fast(x.z - base);
        float part_sum = w * x.weight;
#pragma unroll 1
        for (int d = count; d < 32; d <<= 1) part_sum += __shfl_xor_sync(kAll, part_sum, d);
        sum = fmaf(sum, old, part_sum);
        m = top;
        if (i > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f = __shfl_sync(kAll, old, e);
#pragma unroll
                for (int v = 0; v < NV; ++v) a[e][v] = make_float4(a[e][v].x * f, a[e][v].y * f, a[e][v].z * f, a[e][v].w * f);
            }
        }
        const unsigned on = __ballot_sync(kAll, there);
#pragma unroll 1
        for (int b = 0; b < 32; b += kBatch) {
            if (!(on >> b)) break;
            float4 o[kBatch][NV];
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                // (no branch around a load: each would wait for the one before)
                const float* row = shfl_ptr(x.o, b + e);
                const float* at = wide ? row + 4 * lane : zeros;
#pragma unroll
                for (int v = 0; v < NV; ++v) o[e][v] = *reinterpret_cast<const float4*>(at + 128 * v);
            }
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
                const float f = __shfl_sync(kAll, w, b + e);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float4& y = a[e & 7][v];
                    y = make_float4(fmaf(f, o[e][v].x, y.x), fmaf(f, o[e][v].y, y.y), fmaf(f, o[e][v].z, y.z),
                                    fmaf(f, o[e][v].w, y.w));
                }
            }
        }
    }
    auto add = [](float4& x, const float4& y) { x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w); };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        if (count <= 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) add(a[e][v], a[e + 4][v]);
        if (count <= 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) add(a[e][v], a[e + 2][v]);
        if (count <= 1) add(a[0][v], a[1][v]);
    }
    const float inv = sum == 0.f ? 0.f : reciprocal(sum);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        unsigned char* out = shfl_ptr(row.out, e);
        const float f = __shfl_sync(kAll, inv, e);
        if (e >= count || !out || !wide) continue;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const float4 x = a[e][v];
            *reinterpret_cast<uint2*>(out + 2 * (4 * lane + 128 * v)) =
                make_uint2(f32_to_pair(make_float2(x.x * f, x.y * f), T()), f32_to_pair(make_float2(x.z * f, x.w * f), T()));
        }
    }
    if (lane < count && row.out) {
        const float lse2 = sum == 0.f ? -INFINITY : m + log2f(sum);
        *row.lse = p.base2 ? lse2 : lse2 * kLn2;
    }
}
__device__ __forceinline__ unsigned char* out_row(const PrefixParams& p, int r, int64_t t, int h) {
    return p.o + (int64_t)r * p.o_sn + t * p.o_st + (int64_t)h * p.o_sh;
}
__device__ __forceinline__ float* out_lse(const PrefixParams& p, int r, int64_t t, int h) {
    return p.lse + (int64_t)r * p.l_sn + t * p.l_st + (int64_t)h * p.l_sh;
}

// ---------------------------------------------------------------------------
// slim own parts
// ---------------------------------------------------------------------------

__device__ __noinline__ int share_out_of_line(int n, int r, int N) { return rank_share(n, r, N); }

// Item (request, rank, KV head) by 1 << wlog warps of the CTA, its group number `group`.
template <typename T, int D>
__device__ __forceinline__ void slim_part(const PrefixParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                          const ChunkPartials& ws, int tpi, int rows, int ctas, int item, int group,
                                          int wlog, int ring_bytes, uint8_t* smem, SlimBars* bars, Parts* parts) {
    using S = Slim<D>;
    constexpr int WD = S::WD, DW = S::DW, NB = D / 64;
    __shared__ float row_m[64], row_l[64];
    __shared__ unsigned poisons[4][4];  // by group: tokens of the masked tiles whose V row is not finite
    const int wpi = 1 << wlog, threads = 32 << wlog;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & (wpi - 1), g = lane >> 2, c = lane & 3;
    const int tid = 32 * warp + lane;  // within the group
    // (a barrier for one warp, too: what tests for it would come twice)
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory"); };
    const int b = item / (p.N * p.Hkv), rh = item - b * (p.N * p.Hkv), r = rh / p.Hkv, hkv = rh - r * p.Hkv;
    const Planned q = load_planned(p.slim + 2 * (int64_t)b);
    if (q.n == 0) return;
    bool joined = q.kind == kOwn;
    Planned common;
    common.start = common.n = 0;
    if (joined) common = load_request(p, q.common);
    const int nrows = q.n * p.gq;
    auto seen = [&](int j) { return share_out_of_line(p.causal ? q.L - q.n + j + 1 : q.L, r, p.N); };
    const int lim0 = seen(0), lim_last = q.n == 1 ? lim0 : seen(q.n - 1);
    const int64_t table = table_at(p, q, r, b);
    // row blocks (1 << rlog), and rings of tiles between them, each for a block's or all blocks' warps
    const int xlog = wlog - (WD - 1), wx_all = 1 << xlog;
    const int rlog = min(nrows <= 16 ? 0 : nrows <= 32 ? 1 : 2, xlog), wt = wx_all >> rlog;
    const int wd = warp >> xlog, wx = warp & (wx_all - 1), blk = wx & ((1 << rlog) - 1), first = wx >> rlog;
    const int sharers = WD << rlog, stages = min(sharers * ring_bytes / S::kTile, kMaxStages);
    smem += group * (wpi * ring_bytes);
    uint8_t* const ring = smem + first * (sharers * ring_bytes);
    const int set = group * wx_all + first;
    float* const rm = row_m + group * (16 * wx_all);
    float* const rl = row_l + group * (16 * wx_all);
    unsigned* const poison = poisons[group];
    if (lane == 0 && blk == 0 && wd == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&bars->full[set][i], 1);
            mbar_init(&bars->empty[set][i], sharers);
        }
        fence_mbar_init();
    }
    if (tid < 4) poison[tid] = 0u;
    // the rows' queries as A operands
    unsigned qf[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int row = 16 * blk + g + 8 * e, j = row / p.gq;
        const bool real = row < nrows;
        const unsigned* at = reinterpret_cast<const unsigned*>(
            p.q + (int64_t)(q.start + (real ? j : 0)) * p.q_st + (int64_t)(hkv * p.gq + (real ? row - j * p.gq : 0)) * p.q_sh) + c;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            qf[x][e] = real ? __ldg(at + 8 * x) : 0u;
            qf[x][2 + e] = real ? __ldg(at + 8 * x + 4) : 0u;
        }
    }
    // scores enter with the scale's sign, so that the maximum is that of the scaled ones
    const float sign = p.sm_scale < 0.f ? -1.f : 1.f, qs = fabsf(p.sm_scale) * kLog2e;
    int lim[2] = {lim0, lim0};
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * blk + g + 8 * i;
        int x = lim0;
        if (q.n > 1) x = seen(row / p.gq);
        if (row >= nrows) x = 0;
        if (i) lim[1] = x;
        else lim[0] = x;
    }
    sync();
    const int tiles = (lim_last + kTileTokens - 1) / kTileTokens;
    const int mine = max(tiles - first + wt - 1, 0) / wt;  // of this ring
    const int pb = min(1 << p.page_shift, kTileTokens);    // rows of a box: a page, or a tile of one
    const bool loads = blk == 0 && wd == 0;                // this warp fills the ring
    volatile int* abort = &bars->abort;
    auto token = [&](int i) { return kTileTokens * (first + i * wt); };
    // page of the lane's box of tile i (a page outside of the pool reads zeros)
    auto page_at = [&](int i) -> int {
        const int t = token(i) + lane * pb;
        if (i >= mine || lane * pb >= kTileTokens || t >= lim_last) return -1;
        const int pg = __ldg(p.bt + table + (t >> p.page_shift));
        return (unsigned)pg < (unsigned)p.num_pages ? pg : p.num_pages;
    };
    auto load = [&](int i, int s, int page) {
        if (lane == 0)
            mbar_arrive_expect_tx(&bars->full[set][s],
                                  (min(kTileTokens, lim_last - token(i)) + pb - 1) / pb * (pb * 4 * D));
        __syncwarp();
        if (page >= 0) {
            uint8_t* dst = ring + s * S::kTile + lane * pb * 128;
            const int slot = (token(i) + lane * pb) & ((1 << p.page_shift) - 1);
#pragma unroll
            for (int x = 0; x < NB; ++x) {
                tma_load_5d(dst + x * S::kBox, &kmap, &bars->full[set][s], 64 * x, hkv, slot, page, r);
                tma_load_5d(dst + (NB + x) * S::kBox, &vmap, &bars->full[set][s], 64 * x, hkv, slot, page, r);
            }
        }
        __syncwarp();
    };
    int issued = 0;
    if (loads && !p.stall_loads)
#pragma unroll 1
        for (; issued < min(stages, mine); ++issued) load(issued, issued, page_at(issued));
    int page = loads ? page_at(issued) : -1;  // of the next tile to be loaded
    float o[DW / 8][4];
#pragma unroll
    for (int i = 0; i < DW / 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    bool ok = true;
    const uint32_t k_lane = (uint32_t)(((lane & 7) + 8 * (lane >> 4)) * 128), k_xor = (uint32_t)((((lane >> 3) & 1) ^ (lane & 7)) << 4);
    const uint32_t v_lane = (uint32_t)((lane & 15) * 128), v_xor = (uint32_t)(((lane >> 4) ^ (lane & 7)) << 4);
    int s = 0, phase = 0;
#pragma unroll 1
    for (int i = 0; i < mine; ++i) {
        ok = __all_sync(kAll, mbar_wait(&bars->full[set][s], phase, &g_finish_status, DCP_ERR_TIMEOUT, abort));
        if (!ok) break;
        const int t = token(i);
        uint8_t* tile = ring + s * S::kTile;
        const uint32_t kt = smem_u32(tile), vt = kt + (NB + DW / 64 * wd) * S::kBox;
        float x[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            unsigned w[4];
            ldsm4(w, kt + (kk >> 2) * S::kBox + k_lane + (k_xor ^ (32 * (kk & 3))));
            mma16816<T>(x[0], qf[kk], w[0], w[1]);
            mma16816<T>(x[1], qf[kk], w[2], w[3]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int y = 0; y < 4; ++y) x[e][y] *= sign;
        const bool masked = t + kTileTokens > lim0;
        if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (t + 8 * e + 2 * c + (y & 1) >= lim[y >> 1]) x[e][y] = -INFINITY;
            // values of no token are zeroed, and values that some rows may not see made finite: they must not
            // reach those as 0 * inf (warps that share the tile write the same)
#pragma unroll 1
            for (int id = lane; id < kTileTokens * (D / 8); id += 32) {
                const int row = id / (D / 8), u = id % (D / 8);
                uint4* at = reinterpret_cast<uint4*>(tile + (NB + (u >> 3)) * S::kBox + row * 128 + (((u & 7) ^ (row & 7)) << 4));
                if (t + row >= lim_last) {
                    *at = make_uint4(0u, 0u, 0u, 0u);
                } else if (lim0 < lim_last) {
                    const uint4 w = *at;
                    if (pair_nonfinite<T>(w.x) || pair_nonfinite<T>(w.y) || pair_nonfinite<T>(w.z) || pair_nonfinite<T>(w.w)) {
                        *at = make_uint4(pair_finite<T>(w.x), pair_finite<T>(w.y), pair_finite<T>(w.z), pair_finite<T>(w.w));
                        // below 96, as an item's rows are at most 64 tokens' and what they see differs by less
                        const int n = t - (lim0 & ~15) + row;
                        if (n < 128) atomicOr(&poison[n >> 5], 1u << (n & 31));
                    }
                }
            }
            fence_proxy_async_smem();  // before the next copy into the tile
            __syncwarp();
        }
        float mx[2];
        bool grow = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
            grow |= (mx[e] - ref[e]) * qs > kGrow || (ref[e] == -INFINITY && mx[e] > -INFINITY);
        }
        // (a row's maximum has grown only if that of one of its lanes' has)
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(kAll, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(kAll, mx[e], 2));
                // a row moves by its own maximum alone: rows of no query have no say in how others are rounded
                float alpha = 1.f;
                if ((mx[e] - ref[e]) * qs > kGrow || (ref[e] == -INFINITY && mx[e] > -INFINITY)) {
                    alpha = ref[e] == -INFINITY ? 0.f : exp2_fast((ref[e] - mx[e]) * qs);
                    ref[e] = mx[e];
                }
                l[e] *= alpha;
#pragma unroll
                for (int n = 0; n < DW / 8; ++n) {
                    o[n][2 * e] *= alpha;
                    o[n][2 * e + 1] *= alpha;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float m = ref[e] == -INFINITY ? 0.f : ref[e];
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int y = 2 * e; y < 2 * e + 2; ++y) {
                    // (-infinity times a scale of 0 is no weight)
                    x[n][y] = x[n][y] == -INFINITY ? 0.f : exp2_fast(fmaf(x[n][y] - m, qs, kBias<T>));
                    l[e] += x[n][y];
                }
        }
        // weights in the payload type (half a step a term); the row sums take them unrounded
        const unsigned a[4] = {f32_to_pair(make_float2(x[0][0], x[0][1]), T()),
                               f32_to_pair(make_float2(x[0][2], x[0][3]), T()),
                               f32_to_pair(make_float2(x[1][0], x[1][1]), T()),
                               f32_to_pair(make_float2(x[1][2], x[1][3]), T())};
#pragma unroll
        for (int n = 0; n < DW / 16; ++n) {
            unsigned w[4];
            ldsm4_t(w, vt + (n >> 2) * S::kBox + v_lane + (v_xor ^ (32 * (n & 3))));
            mma16816<T>(o[2 * n], a, w[0], w[1]);
            mma16816<T>(o[2 * n + 1], a, w[2], w[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->empty[set][s]);
        if (loads && issued < mine) {  // into the stage that is done with
            ok = __all_sync(kAll, mbar_wait(&bars->empty[set][s], phase, &g_finish_status, DCP_ERR_TIMEOUT, abort));
            if (!ok) break;
            load(issued, s, page);
            page = page_at(++issued);
        }
        if (++s == stages) {
            s = 0;
            phase ^= 1;
        }
    }
    if (!ok && loads && lane == 0) {  // copies still in flight land before the ring's memory goes
        for (int i = max(issued - stages, 0); i < issued; ++i) {
            const uint64_t t0 = global_timer_ns();
            while (!mbar_try_wait(&bars->full[set][i % stages], (i / stages) & 1) && global_timer_ns() - t0 < kWaitLimitNs / 100) {
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
    }
    sync();  // every warp is done with the ring
    // the warps' shares of a row: wt of them, 16 << rlog rows apart
    float* os = reinterpret_cast<float*>(smem);  // [wx_all][16][D]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = 16 * wx + g + 8 * i;
        if (wd == 0 && c == 0) {
            rm[at] = ref[i] == -INFINITY ? -INFINITY : fmaf(ref[i], qs, -kBias<T>);
            rl[at] = l[i];
        }
#pragma unroll
        for (int n = 0; n < DW / 8; ++n)
            *reinterpret_cast<float2*>(os + at * D + DW * wd + 8 * n + 2 * c) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
    }
    sync();
    if ((poison[0] | poison[1] | poison[2] | poison[3]) != 0u) {
        // what the zeroed values give to the rows that do see them, in the unit of a share that has seen something
#pragma unroll 1
        for (int row = tid; row < nrows; row += threads) {
            const int j = row / p.gq;
            const T* qrow = reinterpret_cast<const T*>(p.q + (int64_t)(q.start + j) * p.q_st +
                                                       (int64_t)(hkv * p.gq + row - j * p.gq) * p.q_sh);
            int at = row;
            while (rm[at] == -INFINITY && at + (16 << rlog) < 16 * wx_all) at += 16 << rlog;
            if (rm[at] != -INFINITY)
                add_nonfinite<T, float>(p, r, table, hkv, qrow, lim0 & ~15, poison, 4, seen(j), rm[at], os + at * D);
        }
        sync();
    }
    // what follows reads what the chunk kernel left
    chain_wait();
    joined = joined && q.start >= common.start && q.start + q.n <= common.start + common.n;  // (groups out of order)
    int qt0 = 0;
    if (joined) {
        qt0 = (q.start - common.start) / tpi;
        const int last = q.n == 1 ? qt0 : (q.start + q.n - 1 - common.start) / tpi;
#pragma unroll 1
        for (int k = warp; qt0 + k <= last; k += wpi) {  // two at most
            const ChunkPos x = {q.common, rh, qt0 + k, 0};
            find_parts(ws.pos, ctas, x, &parts[2 * group + k]);
        }
        sync();
    }
#pragma unroll 1
    for (int row0 = warp; row0 < nrows; row0 += 8 * wpi) {
        const int left = (nrows - row0 + wpi - 1) >> wlog;
        const int count = left > 4 ? 8 : left > 2 ? 4 : left;
        const int row = row0 + wpi * (lane & (count - 1));
        const bool real = row < nrows;
        const int j = real ? row / p.gq : 0, h = hkv * p.gq + (real ? row - j * p.gq : 0), tok = q.start + j;
        const int block = joined ? (tok - common.start) / tpi - qt0 : 0;
        const Parts& from = parts[2 * group + block];
        const bool cut = joined && from.n >= 0;
        const int64_t at = cut ? (int64_t)(tok - common.start - (qt0 + block) * tpi) * p.gq + (h - hkv * p.gq)
                               : ((int64_t)r * p.T + tok) * p.H + h;
        JoinRow x;
        x.out = real ? out_row(p, r, tok, h) : nullptr;
        x.lse = out_lse(p, r, tok, h);
        x.parts = !real ? 0 : wt + (!joined ? 0 : cut ? from.n : 1);
        join_rows<T, D>(p, count, x, [&](int n) -> Part {
            if (n < wt) {
                const int share = row + (n * 16 << rlog);
                return {os + share * D, rm[share], rl[share]};
            }
            const int64_t i = cut ? (int64_t)from.slot[n - wt] * rows + at : at;
            return {(cut ? ws.o : p.wo) + i * D, (cut ? ws.lse : p.wl)[i], 1.f};
        });
    }
}

// ---------------------------------------------------------------------------
// the join of the parts that the chunk kernel has computed
// ---------------------------------------------------------------------------

// Range `c` of the chunk kernel: the items of own parts that begin in it and are joined
// or cut; a CTA takes every `slices`-th of their rows' eights.
template <typename T, int D>
__device__ void join_rest(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int c, int slice,
                          int slices, Parts* parts) {
    constexpr int kWarps = kFinishThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the next kernel of the stream waits for this one only: it must not end before the chunk kernel has
    chain_wait();
    if (*p.nothing) return;
    ChunkPos x = ws.pos[c];
    const ChunkPos end = ws.pos[c + 1];
    if (x.b >= p.requests) return;  // common parts follow the requests' own
    if (x.tile > 0) {               // begun in an earlier range
        if (same_item(x, end)) return;
        x = next_item(p, x, tpi);
    }
    while (x.b < p.requests && !(same_item(x, end) && end.tile == 0)) {
        const Planned q = load_request(p, x.b);
        if (q.kind == kAlone && !same_item(x, end)) {
            // written by the chunk kernel itself, as all of its request but what the range's end cuts
            if (x.b == end.b) {
                if (end.tile == 0) return;
                x = end;
                x.tile = 0;
            } else {
                x.rh = p.N * p.Hkv - 1;
                x.qt = (q.n - 1) / tpi;
                x = next_item(p, x, tpi);
                continue;
            }
        }
        const int r = x.rh / p.Hkv, hkv = x.rh % p.Hkv, j0 = x.qt * tpi;
        const int nrows = min(tpi, q.n - j0) * p.gq;
        const bool cut = same_item(x, end);  // (end.tile > 0)
        bool joined = q.kind == kOwn;
        Planned common;
        if (joined) {
            common = load_request(p, q.common);
            joined = q.start >= common.start && q.start + q.n <= common.start + common.n;  // (groups out of order)
        }
        const int qt0 = joined ? (q.start + j0 - common.start) / tpi : 0;
        __syncthreads();  // the item before is done with `parts`
        if (warp == 0) find_parts(ws.pos, ctas, x, &parts[0]);
        else if (joined && warp <= 2) {
            const ChunkPos y = {q.common, x.rh, qt0 + warp - 1, 0};
            find_parts(ws.pos, ctas, y, &parts[warp]);
        }
        __syncthreads();
        const int own_n = parts[0].n < 0 ? 1 : parts[0].n;
#pragma unroll 1
        for (int row0 = (slice * kWarps + warp) * 8; row0 < nrows; row0 += slices * kWarps * 8) {
            const int row = row0 + (lane & 7);
            const bool real = row < nrows;
            const int j = real ? row / p.gq : 0, h = hkv * p.gq + (real ? row - j * p.gq : 0), tok = q.start + j0 + j;
            const int block = joined ? (tok - common.start) / tpi - qt0 : 0;
            const int64_t whole = ((int64_t)r * p.T + tok) * p.H + h;
            const int64_t within = (int64_t)(tok - common.start - (qt0 + block) * tpi) * p.gq + (h - hkv * p.gq);
            JoinRow g;
            g.out = real ? out_row(p, r, tok, h) : nullptr;
            g.lse = out_lse(p, r, tok, h);
            g.parts = !real ? 0 : own_n + (!joined ? 0 : parts[1 + block].n < 0 ? 1 : parts[1 + block].n);
            join_rows<T, D>(p, 8, g, [&](int n) -> Part {
                const bool own = n < own_n;
                const Parts& from = parts[own ? 0 : 1 + block];
                if (from.n < 0) {  // (own rows lie behind the common ones)
                    const int64_t i = whole + (own ? (int64_t)p.N * p.T * p.H : 0);
                    return {p.wo + i * D, p.wl[i], 1.f};
                }
                const int64_t i = (int64_t)from.slot[own ? n : n - own_n] * rows + (own ? row : within);
                return {ws.o + i * D, ws.lse[i], 1.f};
            });
        }
        if (cut) break;  // the range ends inside it
        x = next_item(p, x, tpi);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFinishThreads, D == 256 ? 2 : 3)
    prefix_finish_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ PrefixParams p, const __grid_constant__ ChunkPartials ws, int tpi, int rows, int ctas, int blocks, int wlog,
                         int ring_bytes, int slices) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Parts parts[8];
    __shared__ SlimBars bars;
    if ((int)blockIdx.x < blocks) {
        if (threadIdx.x == 0) bars.abort = 0;
        __syncthreads();
        const int group = (int)(threadIdx.x >> 5) >> wlog;
        const int item = (int)blockIdx.x * (4 >> wlog) + group;
        if (item < p.requests * p.N * p.Hkv)
            slim_part<T, D>(p, kmap, vmap, ws, tpi, rows, ctas, item, group, wlog, ring_bytes, smem, &bars, parts);
    } else {
        const int k = blockIdx.x - blocks;
        join_rest<T, D>(p, ws, tpi, rows, ctas, k / slices, k % slices, slices, parts);
    }
}

template <typename T, int D>
cudaError_t launch(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, cudaStream_t stream) {
    const auto kernel = prefix_finish_kernel<T, D>;
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv;
    const int wpi = p.slim_warps;
    const int64_t blocks = p.slim_rows ? (items + 4 / wpi - 1) / (4 / wpi) : 0;
    const int ring = blocks > 2 * device_sm_count() ? Slim<D>::kRingMany : Slim<D>::kRingFew, smem = 4 * ring + 1024;
    // the shared-memory opt-in is the function's on the device, not the call's: always that of the larger ring, as
    // another host thread's call may come between this line and the launch
    constexpr int most = 4 * (Slim<D>::kRingMany > Slim<D>::kRingFew ? Slim<D>::kRingMany : Slim<D>::kRingFew) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    const int slices = 4;
    // starts as soon as an SM is free of the chunk kernel: slim parts need nothing of its results until their join
    const CUtensorMap* maps = static_cast<const CUtensorMap*>(p.slim_maps);
    return launch_chained(kernel, (unsigned)(blocks + ctas * slices), kFinishThreads, smem, stream, maps[0], maps[1],
                          p, ws, tpi, rows, ctas, (int)blocks, wpi == 4 ? 2 : wpi - 1, ring, slices);
}

template <typename T>
cudaError_t launch_d(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, cudaStream_t stream) {
    switch (p.D) {
        case 64: return launch<T, 64>(p, ws, tpi, rows, ctas, stream);
        case 128: return launch<T, 128>(p, ws, tpi, rows, ctas, stream);
        case 256: return launch<T, 256>(p, ws, tpi, rows, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

// Boxes of 64 columns of a head and the rows of a tile, or of a page if that is shorter.
bool page_maps(const PrefixParams& p, int dtype, CUtensorMap* maps) {
    const EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const CUtensorMapDataType dt = dtype == DCP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // a dimension of extent 1 is never stepped over: give it a nominal stride
    auto stride = [](int64_t extent, int64_t bytes) -> cuuint64_t { return (cuuint64_t)(extent > 1 ? bytes : 256); };
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    const int64_t rows = (int64_t)1 << p.page_shift;
    for (int m = 0; m < 2; ++m) {
        const int64_t st = m ? p.v_st : p.k_st, sh = m ? p.v_sh : p.k_sh, sp = m ? p.v_sp : p.k_sp;
        const cuuint64_t dims[5] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)rows, (cuuint64_t)p.num_pages,
                                    (cuuint64_t)p.N};
        const cuuint64_t strides[4] = {stride(p.Hkv, sh), stride(rows, st), stride(p.num_pages, sp),
                                       stride(p.N, m ? p.v_sn : p.k_sn)};
        const cuuint32_t box[5] = {64, 1, (cuuint32_t)(rows < kTileTokens ? rows : kTileTokens), 1, 1};
        if (enc(&maps[m], dt, 5, m ? p.v : p.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    return true;
}

}  // namespace

// Warps of an item: alone, a warp streams longest for the set-up it pays; with fewer items
// than warps fit at once they share its tiles.  Items of more than 16 rows want a warp for
// each 16.  An own part is slim up to the rows of its warps, and up to as many tokens of a
// rank as keep them from outlasting the others: with fewer items, a long part is better
// cut over the SMs.
void slim_limits(PrefixParams& p, int dtype, void* maps) {
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv, sms = device_sm_count();
    const int64_t drafts = ((int64_t)p.T + p.requests - 1) / p.requests;  // new tokens of a request, about
    int warps = items >= 6 * sms ? 1 : items >= 3 * sms ? 2 : 4;
    if (drafts * p.gq > 16) warps = 4;
    if (p.D == 256 && warps < 2) warps = 2;  // a row's columns are two warps'
    p.slim_warps = warps;
    p.slim_rows = 16 * warps / (p.D == 256 ? 2 : 1);
    const int64_t tokens = 512 * (1 + 2 * items / (3 * sms));
    p.slim_tokens = (int)(tokens < 8192 ? tokens : 8192);
    // boxes hold whole 8-row swizzle atoms, and a tensor map describes the pools: without, the chunk kernel takes all
    if (p.page_shift < 3 || !page_maps(p, dtype, static_cast<CUtensorMap*>(maps))) p.slim_rows = 0;
    p.slim_maps = maps;
    // DCP_TEST_STALL_LOADS=1 (tests of the failure path only): no loads are issued, so the first wait on them runs out
    const char* stall = getenv("DCP_TEST_STALL_LOADS");
    p.stall_loads = stall && stall[0] == '1';
}

int prefix_finish_status(bool clear) {
    int s = 0;
    if (cudaMemcpyFromSymbol(&s, g_finish_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && s) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_finish_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return s;
}

cudaError_t launch_prefix_finish(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                                 cudaStream_t stream) {
    if (ctas > kMaxRanges) return cudaErrorInvalidValue;
    return dtype == DCP_F16 ? launch_d<__half>(p, ws, tpi, rows, ctas, stream)
                            : launch_d<__nv_bfloat16>(p, ws, tpi, rows, ctas, stream);
}

}  // namespace dcp
