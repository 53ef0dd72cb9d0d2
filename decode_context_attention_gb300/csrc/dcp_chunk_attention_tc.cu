// dcp_chunk_attention_tc.cu -- attention of a ragged batch's new tokens over every
// rank's paged cache on the 5th-generation tensor cores: D = 64 or 128, pages
// of at least 8 tokens.
//
// The mathematics is dcp_chunk_attention.cu's: rows (new token, query head of
// the group) over the tiles of 128 tokens they see, one pass, an online softmax
// in base 2.  Per tile and 128 rows two products of 128 x 128 x D:
//     S = Q K^T into tensor memory;  P = 2^(S - m) back into S's columns as 16-bit
//     pairs;  O += P V with P the A operand from tensor memory, V read MN-major.
//
// One persistent CTA per SM (the ranges of dcp_chunk.cuh), two stages of 128
// rows, each with its own S / P (128 columns) and O (D columns), so that the
// tensor core works on one stage while the other's exponentials run:
//   * an item of more than 128 rows is a pair of row blocks that share every K and
//     V tile (half the loads of one block alone);
//   * an item of up to 128 rows (single new tokens, drafts) takes alternate tiles
//     to the two stages, whose results are joined at the end: the loads of a
//     long cache then stream without waiting for a tile's softmax.
// Warps 0-3 and 4-7: the softmax of stage 0 and 1, a thread a row, so maxima and
// sums need no exchange.  Warp 8: TMA (Q and the K / V tiles into a ring, a box
// per page).  Warp 9 issues the MMAs.  Warp 10: masked tiles: V rows
// past the last visible token are zeroed, and values that are not finite (0
// times infinity would reach rows that must not see them; they are added to
// the rows that do see them at the end).
// The reference maximum moves only when a row's maximum grows by more than 2^8,
// so O is rarely rescaled; P then reaches 2^8, which a 16-bit type holds and
// fp32 sums do too.  P is rounded to the payload type, half a step per term (fp16:
// and at least 2^-32 of the row's largest term); the row sums use it unrounded.  The
// output differs from that of an unrounded P by 2.6e-3 of its norm in bf16 and 2.9e-4
// in fp16 (from 64 bits by 2.3e-3 and 2.7e-4; its own rounding is 1.7e-3 and 2.1e-4).  A second product with what the rounding
// leaves, for items of one row block, brings it to 1.6e-4 in bf16 and costs every item:
// drafts 239 instead of 200 us, 2048 over 8192 386 instead of 352 (the pairs' loop
// shares the registers and the instruction cache); not taken.
// Warp 11 hands out the parts of the CTA's range, computed ahead of everyone.
// Waits are bounded (1 s, or 1 s in which no load is issued): one that runs out records
// DCP_ERR_TIMEOUT.
// Measured (bf16, 32 query heads over 4, D = 128): 4096 new tokens over 32768, 4
// ranks: 1403 to 1437 us, 1.46 PFLOP/s (0.77 of cuBLAS's burst, 0.86 of its rate under
// the power cap); 2048 over 8192: 352 us.  The tensor core is busy 60% of the active
// cycles, the multi-function unit 30%: a stage's chain (scores to registers, exponentials, P's store, two
// products; 3100 cycles a pair of tiles) is longer than the other stage's
// products, and there is no third stage in 512 columns.
// Four new tokens of 32 requests of 16384: 200 us, 5.4 TB/s (159 us at the copy
// rate), bound by the ends of items, where the ring runs dry.  At D = 64 a tile's chain
// is as long and its products half as long: 2048 over 8192 291 us.
// What the loops of all warps run has to fit the instruction cache, and the issuing
// warps have 56 registers: long waits are out of line and descriptors are made where
// they are used (chunk 373 -> 355 us, drafts 211 -> 199 us).
#include <cuda.h>
#include <math.h>
#include <stdlib.h>

#include <type_traits>

#include "dcp_chunk.cuh"
#include "dcp_mma.cuh"
#include "dcp_sm100_warp.cuh"

namespace dcp {

using namespace sm100;

namespace {

constexpr int kTT = 128;        // tokens of a tile
constexpr int kM = 128;         // rows of a stage
constexpr int kThreadsTc = 384;
constexpr int kChunkB = 128 * 128;  // 64 columns of 128 rows
constexpr int kMisc = 2048;
// A row's weights are 2^(s - m + kBias), m the reference maximum, which moves when the
// row's maximum has passed it by more than kGrow powers of two.  fp16's smallest normal
// is 2^-14: beside a largest weight of 1 the weights of a long tail lose bits from
// there on and are gone below 2^-25, while the row sum keeps them.  The bias uses the
// room above, up to 2^15 with the lag, and cancels in O; the reference is kept less
// the bias, so that a log-sum-exp is the reference plus log2 of the sum as without it.
// A smaller lag leaves more room (kGrow 4: bias 11) but rescales O more often: 355
// against 398 us (2048 over 8192, fp16), 1410 against 1561 (4096 over 32768).
template <typename T>
struct PRange {
    static constexpr float kGrow = 8.f, kBias = 0.f;
};
template <>
struct PRange<__half> {
    static constexpr float kGrow = 8.f, kBias = 7.f;
};
// 2^(s qscale - m) takes one fused step, exact but for one rounding; m itself is
// rounded, which moves a row's weights all alike and its log-sum-exp back, and
// is harmless while m's rounding error (2^-24 |m|) is small.  Beyond this the
// difference of the scores is taken first.
constexpr float kFar = 65536.f;
constexpr unsigned kAllLanes = 0xffffffffu;
constexpr uint32_t kColO = 256;
constexpr uint32_t kCols = 512;
constexpr int kSegs = 3;
constexpr int kPoison = 8;      // per-item records of tokens with non-finite values

__device__ int g_chunk_status;  // first bounded wait that ran out (0 if none)

template <int D>
struct TcShape {
    static constexpr int kTileBytes = (D / 64) * kChunkB;
    // a ring of 5 tiles of 32 KB or 8 of 16 KB beside two Q blocks
    static constexpr int kSlots = D == 128 ? 5 : 8;
    static constexpr int kSmem = (2 + kSlots) * kTileBytes + kMisc + 1024;
};

struct TcBars {
    uint64_t full[8], empty[8];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2], pv_done[2];
    uint64_t v_clean[8];      // by ring slot: the masked tile in it is clean
    uint64_t x_full, x_done;  // an item of one row block: stage 1's sums written, its O read
    uint64_t mma_done;
    uint32_t tmem_base;
    int state[2];             // abort; ring positions whose loads are under way
    unsigned poison[kPoison][12];  // 3 masked tiles of 128 tokens
    float xm[kM], xl[kM];
    alignas(16) ChunkPos range[2];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    alignas(16) int4 seg[kSegs][4];  // the CTA's parts, as warp 11 hands them out
};
static_assert(sizeof(TcBars) <= kMisc, "misc region too small");

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// A volatile read from shared memory: the compiler keeps no copy of it.
__device__ __forceinline__ int4 ld_shared4(const int4* at) {
    int4 x;
    asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(smem_u32(at)));
    return x;
}
__device__ __forceinline__ ChunkSeg read_seg(const int4* at) {
    const int4 a = ld_shared4(at), b = ld_shared4(at + 1), c = ld_shared4(at + 2), d = ld_shared4(at + 3);
    ChunkSeg s;
    s.b = a.x; s.r = a.y; s.hkv = a.z; s.row0 = a.w;
    s.nrows = b.x; s.j0 = b.y; s.t0 = b.z; s.t1 = b.w;
    s.lim0 = c.x; s.lim_last = c.y; s.slot = c.z; s.q.n = c.w;
    s.q.L = d.x; s.q.start = d.y;
    return s;
}
// P of the 32 scores v[OFF ..], 2^(s qscale + off), as 16 columns of pairs at tP; its sum is added to l2.
template <typename T, int OFF>
__device__ __forceinline__ void exp_store(const uint32_t (&v)[128], uint32_t tP, Pair qs2,
                                          Pair off2, Pair (&l2)[2]) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 f = unpack2(fma2(pack2(v[OFF + 2 * e], v[OFF + 2 * e + 1]), qs2, off2));
        const float2 pr = make_float2(exp2_fast(f.x), exp2_fast(f.y));
        add2(l2[e & 1], pack2f(pr.x, pr.y));
        w[e] = f32_to_pair(pr, T());
    }
    tmem_st16(tP, w);
}

// Waits for a part, not for a tile, last as long as the cache is long (a second at some
// 85 million tokens of a part): their limit counts the time in which no load is issued.
struct Moving {
    int seen = -1;
    uint64_t since = 0;
    __device__ bool stalled(int issued) {
        const uint64_t now = global_timer_ns();
        if (issued != seen) {
            seen = issued;
            since = now;
        }
        return now - since > kWaitLimitNs;
    }
};
// state: TcBars::state.  (Out of line it costs the mixed batch 2%.)
__device__ __forceinline__ bool wait_part(uint64_t* bar, uint32_t parity, volatile int* state) {
    if (mbar_try_wait(bar, parity)) return true;
    Moving m;
    while (!mbar_try_wait(bar, parity)) {
        if (state[0]) return false;
        if (m.stalled(state[1])) {
            atomicCAS(&g_chunk_status, 0, DCP_ERR_TIMEOUT);
            state[0] = 1;
            return false;
        }
    }
    return true;
}
// mbar_wait with its long path out of line: the loops around it fit the instruction cache.
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* state) {
    return mbar_wait(bar, parity, &g_chunk_status, DCP_ERR_TIMEOUT, state);
}
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity, volatile int* state) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, state);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsTc, 1)
    chunk_attention_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                              const __grid_constant__ CUtensorMap vmap, const ChunkParams p, const ChunkPartials ws,
                              const int tpi) {
    using S = TcShape<D>;
    constexpr int kSlots = S::kSlots, kTileBytes = S::kTileBytes;
    constexpr int NCH = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = smem + 2 * kTileBytes;
    TcBars* bar = reinterpret_cast<TcBars*>(ring + kSlots * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tj = tpi / 2;        // new tokens of a row block
    const int rblk = tj * p.gq;    // its rows (at most 128)

    // the Q blocks are not in use yet
    find_range<kThreadsTc>(p, tpi, tj, kTT, ws.pos, reinterpret_cast<int64_t*>(smem), bar->range);
    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
            mbar_init(&bar->v_clean[s], 1);
        }
        for (int s = 0; s < kSegs; ++s) {
            mbar_init(&bar->seg_full[s], 1);
            mbar_init(&bar->seg_empty[s], 11);  // warps 0 to 10
        }
        for (int u = 0; u < 2; ++u) {
            mbar_init(&bar->q_full[u], 1);
            mbar_init(&bar->q_empty[u], 1);
            mbar_init(&bar->s_full[u], 1);
            mbar_init(&bar->p_full[u], 4);
            mbar_init(&bar->pv_done[u], 1);
        }
        mbar_init(&bar->x_full, 4);
        mbar_init(&bar->x_done, 4);
        mbar_init(&bar->mma_done, 1);
        bar->state[0] = bar->state[1] = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&bar->tmem_base, kCols);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&qmap);
        tma_prefetch_map(&kmap);
        tma_prefetch_map(&vmap);
    }
    fence_proxy_async_smem();  // the range's scratch is overwritten by copies
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    volatile int* abort = bar->state;
    int* status = &g_chunk_status;
    // the k-th part of this CTA's range, from warp 11; false behind the last one
    auto get_seg = [&](int k, ChunkSeg* g) -> bool {
        if (!__all_sync(kAllLanes, mbar_wait(&bar->seg_full[k % kSegs], (k / kSegs) & 1, status, DCP_ERR_TIMEOUT, abort)))
            return false;
        *g = read_seg(bar->seg[k % kSegs]);
        return g->b >= 0;
    };
    auto release_seg = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->seg_empty[k % kSegs]);
    };
    bool issued_any = false;

    if (warp >= 8) {
        regs_dec<56>();
        if (warp == 8) {
            // ------------------------------------------------------------ TMA
            const int pb = min(1 << p.page_shift, kTT);  // rows of a box: a page, or a tile of one
            int pos = 0, qn[2] = {0, 0};
            bool ok = !p.stall_loads;
            ChunkSeg g;
            for (int seg = 0; ok && get_seg(seg, &g); ++seg) {
                release_seg(seg);
                const int n = g.t1 - g.t0;
                const bool pair = g.nrows > rblk;
                auto load_q = [&](int u) -> bool {
                    int go = 1;
                    if (lane == 0) {
                        if (qn[u] > 0)
                            go = wait_short(&bar->q_empty[u], (qn[u] - 1) & 1, abort);
                        if (go) {
                            mbar_arrive_expect_tx(&bar->q_full[u], (uint32_t)(NCH * rblk * 128));
                            for (int c = 0; c < NCH; ++c)
                                tma_load_3d(smem + u * kTileBytes + c * kChunkB, &qmap, &bar->q_full[u], 64 * c,
                                            g.hkv * p.gq, g.row0 + (pair ? u * tj : 0));
                        }
                    }
                    ++qn[u];
                    return __shfl_sync(kAllLanes, go, 0);
                };
                auto load_tile = [&](int i, const CUtensorMap* map) -> bool {
                    const int s = pos % kSlots;
                    const int tb = (g.t0 + i) * kTT;
                    const int nseg = (min(kTT, g.lim_last - tb) + pb - 1) / pb;
                    int pg = 0;
                    if (lane < nseg) {  // entries of tokens that exist only
                        pg = __ldg(p.bt + (int64_t)g.r * p.bt_sn + (int64_t)g.b * p.bt_sb +
                                   ((tb + lane * pb) >> p.page_shift));
                        if ((unsigned)pg >= (unsigned)p.num_pages) pg = p.num_pages;  // reads zeros
                    }
                    int go = 1;
                    if (lane == 0) {
                        if (pos >= kSlots)
                            go = wait_short(&bar->empty[s], (pos / kSlots - 1) & 1, abort);
                        if (go) {
                            mbar_arrive_expect_tx(&bar->full[s], (uint32_t)(NCH * nseg * pb * 128));
                            __threadfence_block();
                            abort[1] = pos + 1;
                        }
                    }
                    if (!__shfl_sync(kAllLanes, go, 0)) return false;
                    if (lane < nseg) {
                        uint8_t* dst = ring + s * kTileBytes + lane * pb * 128;
                        const int slot = (tb + lane * pb) & ((1 << p.page_shift) - 1);
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            tma_load_5d(dst + c * kChunkB, map, &bar->full[s], 64 * c, g.hkv, slot, pg, g.r);
                    }
                    __syncwarp();
                    ++pos;
                    return true;
                };
                if (pair) {
                    if (n > 0) ok = load_q(0) && load_tile(0, &kmap) && load_q(1) && load_tile(0, &vmap);
                    for (int i = 1; ok && i < n; ++i) ok = load_tile(i, &kmap) && load_tile(i, &vmap);
                } else {
                    if (n > 0) ok = load_q(0) && load_tile(0, &kmap);
                    if (ok && n > 1) ok = load_q(1) && load_tile(1, &kmap);
                    for (int i = 0; ok && i < n; ++i) {
                        ok = load_tile(i, &vmap);
                        if (ok && i + 2 < n) ok = load_tile(i + 2, &kmap);
                    }
                }
            }
            // copies still in flight (only after an abort) land before the CTA ends
            if (lane == 0) {
                for (int j = max(0, pos - kSlots); j < pos; ++j) {
                    const uint64_t t = global_timer_ns();
                    while (!mbar_try_wait(&bar->full[j % kSlots], (j / kSlots) & 1) &&
                           global_timer_ns() - t < kWaitLimitNs) {
                    }
                }
                for (int u = 0; u < 2 && *abort; ++u) {
                    const uint64_t t = global_timer_ns();
                    while (qn[u] > 0 && !mbar_try_wait(&bar->q_full[u], (qn[u] - 1) & 1) &&
                           global_timer_ns() - t < kWaitLimitNs / 100) {
                    }
                }
            }
        } else if (warp == 9) {
            // ------------------------------------------------------------ MMA
            // the whole warp runs along, its leader issues
            constexpr bool kBf16 = !std::is_same<T, __half>::value;
            const uint32_t idesc_s = idesc_f16(kM, kTT, kBf16, 0, 0);
            const uint32_t idesc_o = idesc_f16(kM, D, kBf16, 0, 1);
            const uint32_t tm = __shfl_sync(kAllLanes, tmem, 0);
            const uint32_t qa = __shfl_sync(kAllLanes, smem_u32(smem), 0);
            const uint32_t ra = qa + 2 * kTileBytes;
            int base = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
            unsigned cleaned = 0u;  // phase of v_clean by slot
            bool ok = true;
            ChunkSeg g;
            for (int seg = 0; ok && get_seg(seg, &g); ++seg) {
                release_seg(seg);
                int n, mtile;
                bool pair;
                {
                    n = __shfl_sync(kAllLanes, g.t1 - g.t0, 0);
                    pair = __shfl_sync(kAllLanes, g.nrows > rblk ? 1 : 0, 0) != 0;
                    mtile = __shfl_sync(kAllLanes, g.lim0 / kTT - g.t0, 0);  // masked from here on, within the part
                }
                // ring positions of a tile's K and V
                auto pos_k = [&](int i) { return base + (pair ? 2 * i : (i < 2 ? i : 2 * i - 1)); };
                auto pos_v = [&](int i) { return base + (pair ? 2 * i + 1 : (i < n - 1 ? 2 * i + 2 : 2 * n - 1)); };
                auto wait = [&](uint64_t* b, int parity) -> bool {
                    return __all_sync(kAllLanes, wait_short(b, parity & 1, abort));
                };
                auto issue_s = [&](int u, int i, bool release, bool last) -> bool {
                    const int j = pos_k(i), s = j % kSlots;
                    if (!wait(&bar->full[s], j / kSlots)) return false;
                    tc_fence_after();
                    const uint64_t da = smem_desc(qa + u * kTileBytes, 16, 1024, kSwizzle128B);
                    const uint64_t db = smem_desc(ra + s * kTileBytes, 16, 1024, kSwizzle128B);
#pragma unroll
                    for (int c = 0; c < NCH; ++c)  // 64 elements of D a time: 16 are 32 bytes of a swizzled row
                        mma_ss4_warp<2, 2>(tm + kM * u, (uint32_t)da + c * (kChunkB >> 4), (uint32_t)(da >> 32),
                                           (uint32_t)db + c * (kChunkB >> 4), (uint32_t)(db >> 32), idesc_s, c > 0);
                    mma_commit_warp(&bar->s_full[u]);
                    if (release) mma_commit_warp(&bar->empty[s]);
                    if (last) mma_commit_warp(&bar->q_empty[u]);
                    issued_any = true;
                    return true;
                };
                auto issue_o = [&](int u, int i, bool begin, bool clean, bool release) -> bool {
                    const int j = pos_v(i), s = j % kSlots;
                    if (!wait(&bar->full[s], j / kSlots)) return false;
                    if (clean && i >= mtile) {
                        if (!wait(&bar->v_clean[s], (int)(cleaned >> s))) return false;
                        cleaned ^= 1u << s;
                    }
                    if (!wait(&bar->p_full[u], pn[u])) return false;
                    ++pn[u];
                    tc_fence_after();
                    const uint64_t dv = smem_desc(ra + s * kTileBytes, kChunkB, 1024, kSwizzle128B);
#pragma unroll
                    for (int c = 0; c < kTT / 64; ++c)  // 16 tokens are 8 columns of P and 2 KB of V
                        mma_ts4_warp<8, 128>(tm + kColO + D * u, tm + kM * u + 32 * c, (uint32_t)dv + 512 * c,
                                             (uint32_t)(dv >> 32), idesc_o, !begin || c > 0);
                    mma_commit_warp(&bar->pv_done[u]);
                    if (release) mma_commit_warp(&bar->empty[s]);
                    return true;
                };
                if (pair) {
                    if (n > 0)
                        ok = wait(&bar->q_full[0], qn[0]++) && issue_s(0, 0, false, n == 1) &&
                             wait(&bar->q_full[1], qn[1]++) && issue_s(1, 0, true, n == 1);
                    for (int i = 0; ok && i < n; ++i) {
                        ok = issue_o(0, i, i == 0, true, false);
                        if (ok && i + 1 < n) ok = issue_s(0, i + 1, false, i + 2 == n);
                        if (ok) ok = issue_o(1, i, i == 0, false, true);
                        if (ok && i + 1 < n) ok = issue_s(1, i + 1, true, i + 2 == n);
                    }
                } else {
                    if (n > 0) ok = wait(&bar->q_full[0], qn[0]++) && issue_s(0, 0, true, n <= 2);
                    if (ok && n > 1) ok = wait(&bar->q_full[1], qn[1]++) && issue_s(1, 1, true, n <= 3);
                    for (int i = 0; ok && i < n; i += 2) {
                        ok = issue_o(0, i, i == 0, true, true);
                        if (ok && i + 2 < n) ok = issue_s(0, i + 2, true, i + 4 >= n);
                        if (ok && i + 1 < n) ok = issue_o(1, i + 1, i == 0, true, true);
                        if (ok && i + 3 < n) ok = issue_s(1, i + 3, true, i + 5 >= n);
                    }
                }
                base += 2 * n;
            }
            if (issued_any) mma_commit_warp(&bar->mma_done);
        } else if (warp == 10) {
            // -------------------------------------------- V of the masked tiles
            int base = 0;
            bool ok = true;
            ChunkSeg g;
            // this warp passes over parts without masked tiles, ahead of everyone: the next
            // ones come when the first of them is done
            auto next_seg = [&](int k) -> bool {
                return __all_sync(kAllLanes, wait_part(&bar->seg_full[k % kSegs], (k / kSegs) & 1, abort)) &&
                       get_seg(k, &g);
            };
            for (int seg = 0; ok && next_seg(seg); ++seg) {
                release_seg(seg);
                const int n = g.t1 - g.t0;
                const bool pair = g.nrows > rblk;
                const int m0 = g.lim0 / kTT;
                unsigned* poison = bar->poison[seg & (kPoison - 1)];
                if (lane < 12) poison[lane] = 0u;
                __syncwarp();
                for (int t = max(m0, g.t0); ok && t < g.t1; ++t) {
                    const int i = t - g.t0;
                    const int j = base + (pair ? 2 * i + 1 : (i < n - 1 ? 2 * i + 2 : 2 * n - 1)), s = j % kSlots;
                    // this warp does not wait for every tile, so the slot's barrier may still
                    // be phases behind: its parity means something once the load is under
                    // way (and the slot cannot pass on before this tile is clean)
                    Moving m;
                    for (int got; (got = abort[1]) <= j && !*abort;) {
                        __nanosleep(200);
                        if (m.stalled(got)) {
                            atomicCAS(status, 0, DCP_ERR_TIMEOUT);
                            *abort = 1;
                        }
                    }
                    __threadfence_block();
                    ok = !__any_sync(kAllLanes, *abort != 0) &&
                         __all_sync(kAllLanes,
                                    wait_short(&bar->full[s], (j / kSlots) & 1, abort));
                    if (!ok) break;
                    uint8_t* tile = ring + s * kTileBytes;
                    // 16 bytes a lane, 4 rows of 128 bytes a step
                    const int live = min(max(g.lim_last - t * kTT, 0), kTT);  // rows from here on are no one's
                    uint8_t* mine = tile + (lane >> 3) * 128 + (lane & 7) * 16;
                    for (int r4 = live & ~3; r4 < kTT; r4 += 4) {
                        if (r4 + (lane >> 3) < live) continue;
#pragma unroll
                        for (int c = 0; c < NCH; ++c)
                            *reinterpret_cast<uint4*>(mine + c * kChunkB + r4 * 128) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    if (g.lim0 < g.lim_last) {  // rows of the item differ in what they see
                        for (int r4 = 0; r4 < live; r4 += 16) {
                            uint4 v[4 * NCH];
#pragma unroll
                            for (int e = 0; e < 4 * NCH; ++e)
                                v[e] = *reinterpret_cast<const uint4*>(mine + (e >> 2) * kChunkB +
                                                                       min(r4 + 4 * (e & 3), kTT - 4) * 128);
#pragma unroll
                            for (int e = 0; e < 4 * NCH; ++e) {
                                const int row = r4 + 4 * (e & 3) + (lane >> 3);
                                if (row < live && (pair_nonfinite<T>(v[e].x) || pair_nonfinite<T>(v[e].y) ||
                                                   pair_nonfinite<T>(v[e].z) || pair_nonfinite<T>(v[e].w))) {
                                    *reinterpret_cast<uint4*>(mine + (e >> 2) * kChunkB + (row & ~3) * 128) =
                                        make_uint4(pair_finite<T>(v[e].x), pair_finite<T>(v[e].y),
                                                   pair_finite<T>(v[e].z), pair_finite<T>(v[e].w));
                                    atomicOr(&poison[4 * (t - m0) + (row >> 5)], 1u << (row & 31));
                                }
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->v_clean[s]);
                }
                base += 2 * n;
            }
        } else {
            // ------------------------------------------------ the parts, ahead of everyone
            ChunkPos x = bar->range[0];
            const ChunkPos first = x, end = bar->range[1];
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const bool more = x.b < p.B && !(same_item(x, end) && x.tile == end.tile);
                ChunkSeg g;
                g.b = -1;
                if (more) g = load_seg(p, x, first, end, tpi, kTT);
                if (k >= kSegs)
                    ok = __all_sync(kAllLanes, wait_part(&bar->seg_empty[k % kSegs], (k / kSegs - 1) & 1, abort));
                if (!ok) break;
                if (lane == 0) {
                    int4* at = bar->seg[k % kSegs];
                    at[0] = make_int4(g.b, g.r, g.hkv, g.row0);
                    at[1] = make_int4(g.nrows, g.j0, g.t0, g.t1);
                    at[2] = make_int4(g.lim0, g.lim_last, g.slot, g.q.n);
                    at[3] = make_int4(g.q.L, g.q.start, 0, 0);
                    mbar_arrive(&bar->seg_full[k % kSegs]);
                }
                __syncwarp();
                if (!more) break;
                if (same_item(x, end)) x = end;  // its first tiles were the last part
                else x = next_item(p, x, tpi);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<224>();
        const int u = warp >> 2;             // stage
        const int m = tid & 127;             // row of the stage
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int mtok = m / p.gq, hh = m - mtok * p.gq;  // new token of the row block, head of the group
        const uint32_t tS = tmem + kM * u + lanes, tO = tmem + kColO + D * u + lanes;
        const float qscale = p.sm_scale * kLog2e;
        constexpr float kGrow = PRange<T>::kGrow, kBias = PRange<T>::kBias;
        int sn = 0, vn = 0, xn = 0;  // phases of s_full and pv_done, exchanges
        bool ok = true;
        auto wait = [&](uint64_t* b, int parity) -> bool {
            return __all_sync(kAllLanes, mbar_wait(b, parity & 1, status, DCP_ERR_TIMEOUT, abort));
        };
        for (int seg = 0; ok; ++seg) {
            int n, mine, step, tile0, lim, lim0;
            bool pair, live;
            {
                ChunkSeg g;
                if (!get_seg(seg, &g)) break;
                n = g.t1 - g.t0;
                pair = g.nrows > rblk;
                mine = pair ? n : (n + 1 - u) / 2;  // tiles of this stage
                step = pair ? 1 : 2;
                tile0 = g.t0 + (pair ? 0 : u);
                const int row = (pair ? u * rblk : 0) + m;
                const bool valid = m < rblk && row < g.nrows;
                lim = valid ? visible(p, g.q, g.j0 + (pair ? u * tj : 0) + mtok, g.r) : 0;
                lim0 = g.lim0;
                live = __any_sync(kAllLanes, valid);
            }
            float mref = -INFINITY, vref = -INFINITY;  // the reference: scaled less kBias, and as a score
            bool far = false;                    // a row of the warp has one beyond kFar
            Pair l2[2] = {0ull, 0ull};
            for (int i = 0; i < mine; ++i) {
                if (!(ok = wait(&bar->s_full[u], sn))) break;
                ++sn;
                const int tb = (tile0 + i * step) * kTT;
                if (live) {
                    tc_fence_after();
                    uint32_t v[128];
                    tmem_ld32<0>(tS, v);
                    tmem_ld32<32>(tS + 32, v);
                    tmem_ld32<64>(tS + 64, v);
                    tmem_ld32<96>(tS + 96, v);
                    tmem_wait_ld();
                    pin(v);
                    if (tb + kTT > lim0) {
                        const int seen = lim - tb;
#pragma unroll
                        for (int c = 0; c < 128; ++c)
                            if (c >= seen) v[c] = 0xff800000u;
                    }
                    float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 128; c += 8) {
                        m0 = max3(m0, __uint_as_float(v[c]), __uint_as_float(v[c + 1]));
                        m1 = max3(m1, __uint_as_float(v[c + 2]), __uint_as_float(v[c + 3]));
                        m2 = max3(m2, __uint_as_float(v[c + 4]), __uint_as_float(v[c + 5]));
                        m3 = max3(m3, __uint_as_float(v[c + 6]), __uint_as_float(v[c + 7]));
                    }
                    const float vt = fmaxf(max3(m0, m1, m2), m3);
                    // rows of no query (of the next request, of the padding, or of none at all) have
                    // no say in how the warp's other rows are rounded; a query's row that sees
                    // nothing (lim 0) has a maximum of -infinity anyway
                    // (the difference of the scores is exact where they are near each other; that of
                    // two scaled maxima is off by more than kGrow from 2^26 on)
                    const bool grow = lim > 0 && (vt - vref) * qscale > kGrow;
                    if (__any_sync(kAllLanes, grow)) {
                        float alpha = 1.f;
                        if (grow) {
                            alpha = mref == -INFINITY ? 0.f : exp2_fast((vref - vt) * qscale);
                            vref = vt;
                            mref = vt * qscale - kBias;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 l = unpack2(l2[e]);
                                l2[e] = pack2f(l.x * alpha, l.y * alpha);
                            }
                        }
                        far = __any_sync(kAllLanes, fabsf(mref) > kFar && mref != -INFINITY);
                        if (i > 0) {  // O holds the tiles before: rescale it once the last of them has landed
                            if (!(ok = wait(&bar->pv_done[u], vn + i - 1))) break;
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * c, o);
                                tmem_wait_ld();
                                pin(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                tmem_st16(tO + 16 * c, o);
                            }
                        }
                    }
                    const float off = far ? kBias : mref == -INFINITY ? 0.f : -mref;
                    if (far) {
                        const float sub = mref == -INFINITY ? 0.f : vref;
#pragma unroll
                        for (int c = 0; c < 128; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) - sub);
                    }
                    const Pair qs2 = pack2f(qscale, qscale), off2 = pack2f(off, off);
                    exp_store<T, 0>(v, tS, qs2, off2, l2);
                    exp_store<T, 32>(v, tS + 16, qs2, off2, l2);
                    exp_store<T, 64>(v, tS + 32, qs2, off2, l2);
                    exp_store<T, 96>(v, tS + 48, qs2, off2, l2);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->p_full[u]);
            }
            if (ok && mine > 0) ok = wait(&bar->pv_done[u], vn + mine - 1);
            vn += mine;
            tc_fence_after();
            add2(l2[0], l2[1]);
            const float2 lp = unpack2(l2[0]);
            float l = lp.x + lp.y;
            // an item of one row block: stage 0 takes what stage 1 has
            float w0 = 1.f, w1 = 0.f;
            if (!pair && ok) {
                if (u == 1) {
                    bar->xm[m] = mref;
                    bar->xl[m] = l;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->x_full);
                    ok = wait(&bar->x_done, xn);
                    tc_fence_after();
                } else {
                    ok = wait(&bar->x_full, xn);
                    tc_fence_after();
                    const float m1 = bar->xm[m], l1 = bar->xl[m];
                    const float mx = fmaxf(mref, m1), z = mx == -INFINITY ? 0.f : mx;
                    w0 = exp2_fast(mref - z);
                    w1 = n > 1 ? exp2_fast(m1 - z) : 0.f;
                    l = l * w0 + (n > 1 ? l1 * w1 : 0.f);
                    mref = mx;
                }
                ++xn;
            }
            // the item again, for where its rows go: held through the tiles it would take
            // the registers of their scores
            const ChunkSeg g = read_seg(bar->seg[seg % kSegs]);
            const int row = (pair ? u * rblk : 0) + m;  // row of the item
            const bool valid = m < rblk && row < g.nrows;
            const int tok = (pair ? u * tj : 0) + mtok;
            // l is 0 only where the row sees nothing (a visible row's largest term is at least 2^kBias); NaN stays NaN
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse2 = l == 0.f ? -INFINITY : mref + log2f(l);
            const bool writes = ok && live && (pair || u == 0);
            const int h = g.hkv * p.gq + hh;
            const int64_t t = g.row0 + tok;
            if (writes) {
                unsigned char* orow = p.o + (int64_t)g.r * p.o_sn + t * p.o_st + (int64_t)h * p.o_sh;
                const int64_t prow = (int64_t)g.slot * (2 * kM) + row;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32<0>(tO + 32 * c, o);
                        tmem_wait_ld();
                        pin(o);
                        const float a = w0 * inv;
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
                        if (!pair && n > 1) {
                            uint32_t o1[32];
                            tmem_ld32<0>(tO + D + 32 * c, o1);
                            tmem_wait_ld();
                            pin(o1);
                            const float b = w1 * inv;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), b, __uint_as_float(o[e])));
                        }
                    }
                    if (valid) {
                        // a row that sees nothing is zero, whatever the accumulator holds
                        if (n == 0 || l == 0.f) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0u;
                        }
                        if (g.slot < 0) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    w[k] = f32_to_pair(make_float2(__uint_as_float(o[8 * e + 2 * k]),
                                                                   __uint_as_float(o[8 * e + 2 * k + 1])), T());
                                *reinterpret_cast<uint4*>(orow + 64 * c + 16 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<uint4*>(ws.o + prow * D + 32 * c + 4 * e) =
                                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                    __syncwarp();
                }
                if (valid) {
                    if (g.slot < 0)
                        p.lse[(int64_t)g.r * p.l_sn + t * p.l_st + (int64_t)h * p.l_sh] = p.base2 ? lse2 : lse2 * kLn2;
                    else
                        ws.lse[prow] = lse2;
                    // what the zeroed values of masked tiles give to the rows that do see them
                    const int mt0 = g.lim0 / kTT;
                    if (g.lim0 < g.lim_last && g.t1 > mt0) {
                        volatile unsigned* mask = bar->poison[seg & (kPoison - 1)];
                        unsigned any = 0u;
#pragma unroll
                        for (int e = 0; e < 12; ++e) any |= mask[e];
                        if (any) {
                            const T* qrow = reinterpret_cast<const T*>(p.q + t * p.q_st + (int64_t)h * p.q_sh);
                            for (int e = 0; e < 3; ++e) {
                                if (g.slot < 0)
                                    add_nonfinite<T, T>(p, g.r, g.b, g.hkv, qrow, (mt0 + e) * kTT,
                                                        (const unsigned*)mask + 4 * e, 4, lim, lse2,
                                                        reinterpret_cast<T*>(orow));
                                else
                                    add_nonfinite<T, float>(p, g.r, g.b, g.hkv, qrow, (mt0 + e) * kTT,
                                                            (const unsigned*)mask + 4 * e, 4, lim, lse2,
                                                            ws.o + prow * D);
                            }
                        }
                    }
                }
            }
            if (!pair && u == 0) {  // stage 1 may go on
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->x_done);
            }
            release_seg(seg);
        }
    }

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        if (lane == 0 && issued_any) {
            // every MMA this CTA issued has completed before its tensor memory goes
            const uint64_t t = global_timer_ns();
            while (!mbar_try_wait(&bar->mma_done, 0) && global_timer_ns() - t < kWaitLimitNs) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

template <typename T, int D>
cudaError_t launch_tc(const ChunkParams& p, const CUtensorMap (&maps)[3], int dtype, cudaStream_t stream) {
    const int ctas = device_sm_count(), tpi = 2 * (kM / p.gq);
    const ChunkPartials ws = chunk_partials_in(p.ws, ctas, 2 * kM, D);
    const void* k = (const void*)chunk_attention_tc_kernel<T, D>;
    // the shared-memory opt-in is a per-device function attribute
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, TcShape<D>::kSmem);
    if (e != cudaSuccess) return e;
    chunk_attention_tc_kernel<T, D>
        <<<ctas, kThreadsTc, TcShape<D>::kSmem, stream>>>(maps[0], maps[1], maps[2], p, ws, tpi);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_chunk_merge(p, ws, tpi, kTT, 2 * kM, ctas, dtype, stream);
}

}  // namespace

size_t chunk_attention_tc_workspace(int D) {
    return D == 64 || D == 128 ? chunk_partials_bytes(device_sm_count(), 2 * kM, D) : 0;
}

bool launch_chunk_attention_tc(const ChunkParams& p, int dtype, cudaStream_t stream, cudaError_t* err) {
    // the maximum of the scaled scores is that of the scores for a positive scale
    // only; boxes hold whole 8-row swizzle atoms.  Where both kernels can run this one
    // takes 199 against 326 us (drafts), 144 against 358 (mixed, D = 64), 353 against
    // 1891 and 1403 against 8085 (chunks), 35 against 41 (32 ragged requests of up to
    // 40 over 500), 12.5 against 13.0 (8 single tokens over 200).  It loses where every
    // request is short, by its fixed part per item: 27 against 15 (64 single tokens over
    // 128), 109 against 47 (256 requests, 2 over 100), 12 against 9.5 (one over 64).
    // The lengths that tell these apart are on the device, where a captured graph
    // follows them; max_seq_len bounds them only
    if ((p.D != 64 && p.D != 128) || !(p.sm_scale > 0.f) || p.page_shift < 3) return false;
    const EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const CUtensorMapDataType dt = dtype == DCP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // a dimension of extent 1 is never stepped over: give it a nominal stride
    auto stride = [](int64_t extent, int64_t bytes) -> cuuint64_t { return (cuuint64_t)(extent > 1 ? bytes : 256); };
    CUtensorMap maps[3];
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    {
        const cuuint64_t dims[3] = {(cuuint64_t)p.D, (cuuint64_t)p.H, (cuuint64_t)p.T};
        const cuuint64_t strides[2] = {stride(p.H, p.q_sh), stride(p.T, p.q_st)};
        const cuuint32_t box[3] = {64, (cuuint32_t)p.gq, (cuuint32_t)(kM / p.gq)};
        if (enc(&maps[0], dt, 3, const_cast<unsigned char*>(p.q), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;
    }
    for (int m = 0; m < 2; ++m) {
        const int64_t rows = (int64_t)1 << p.page_shift;
        const int64_t st = m ? p.v_st : p.k_st, sh = m ? p.v_sh : p.k_sh, sp = m ? p.v_sp : p.k_sp;
        const cuuint64_t dims[5] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)rows, (cuuint64_t)p.num_pages,
                                    (cuuint64_t)p.N};
        const cuuint64_t strides[4] = {stride(p.Hkv, sh), stride(rows, st), stride(p.num_pages, sp),
                                       stride(p.N, m ? p.v_sn : p.k_sn)};
        const cuuint32_t box[5] = {64, 1, (cuuint32_t)(rows < kTT ? rows : kTT), 1, 1};
        if (enc(&maps[1 + m], dt, 5, m ? p.v : p.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return false;  // strides a tensor map cannot describe: the register-tiled kernel takes it
    }
    ChunkParams q = p;
    // DCP_TEST_STALL_LOADS=1 (tests of the failure path only): no loads are
    // issued, so the first wait on them runs out.  Unset in normal use.
    const char* stall = getenv("DCP_TEST_STALL_LOADS");
    q.stall_loads = stall && stall[0] == '1';
    if (p.D == 128)
        *err = dtype == DCP_F16 ? launch_tc<__half, 128>(q, maps, dtype, stream)
                                : launch_tc<__nv_bfloat16, 128>(q, maps, dtype, stream);
    else
        *err = dtype == DCP_F16 ? launch_tc<__half, 64>(q, maps, dtype, stream)
                                : launch_tc<__nv_bfloat16, 64>(q, maps, dtype, stream);
    return true;
}

int chunk_attention_tc_status(bool clear) {
    int s = 0;
    if (cudaMemcpyFromSymbol(&s, g_chunk_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && s) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_chunk_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return s;
}

}  // namespace dcp
