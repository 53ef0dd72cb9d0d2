// dcp_chunk_weights_tc.cu -- the accumulated attention weights of
// dcp_chunk_weights.cu on the 5th-generation tensor cores: D = 64 or 128, pages
// of at least 8 tokens.
//
// With the merged log-sum-exp known a weight is one exponential and a token's sum
// needs no other token, so the product runs transposed, tokens on M:
//     S^T [128 tokens x up to 128 rows] = K_tile . Q_tile^T   (tcgen05, K-major both)
//     acc[token] += sum over rows of 2^(S^T sm_scale log2e - lse2[row])
// and a thread owns a token: its row of S^T comes from tensor memory, the rows'
// log-sum-exps from shared memory (one address for the warp), the sum never
// leaves its registers.  An item is a block of 256 tokens, two tiles of 128 that
// share every tile of queries; it stays in shared memory while the queries pass
// by, so the keys are read once (a decode step: they are all that is read) and a
// chunk's queries are read from L2, 32 KB per 2 x 128 x 128 x D products.
// The items, cut evenly by their number of query tiles, go to one persistent CTA
// per SM; every CTA finds its range itself from the lengths (sums of floors, as
// in the chunk attention).
// Warps 0-15: the sums, four warps for each of the block's two tiles and of the
// two score buffers (query tiles alternate; at the end of an item one of the two
// adds its sum to what the other has written): with eight warps the waits of a
// tile were half its time.  Warp 16: TMA (the next block's keys while this one is
// worked on, a ring of query tiles); warp 17: MMAs; warps 18 and 19: the
// log-sum-exps of the even and the odd query tiles' rows.
// Waits are bounded (1 s): one that runs out records DCP_ERR_TIMEOUT.
// Measured (D = 128, bf16, 32 query heads over 4): one new token of 64 requests of
// 8192 tokens, 4 ranks: 97 us, 5.7 TB/s, bound by the keys' bytes (82 us at the copy
// rate); 2048 new tokens over 16384, 2 ranks: 277 us, 0.93 PFLOP/s: the two tiles'
// 2 x 128 exponentials a row of threads take the multi-function unit as long as
// their products take the tensor core, each is busy under half of the cycles, and
// 256 blocks over 152 CTAs leave a sixth of them idle.
#include <cuda.h>
#include <math.h>
#include <stdlib.h>

#include <type_traits>

#include "dcp_chunk.cuh"
#include "dcp_sm100_warp.cuh"

namespace dcp {

using namespace sm100;

namespace {

constexpr int kM = 128;         // tokens of a tile, and the most query rows of one
constexpr int kThreadsW = 640;
constexpr int kChunkB = 128 * 128;  // 64 columns of 128 rows
constexpr unsigned kAllLanes = 0xffffffffu;

__device__ int g_weights_status;  // first bounded wait that ran out (0 if none)

template <int D>
struct WShape {
    static constexpr int kTileBytes = (D / 64) * kChunkB;
    static constexpr int kQSlots = D == 128 ? 3 : 6;
    static constexpr int kMisc = 2 * kM * 4 + 512;
    static constexpr int kSmem = (4 + kQSlots) * kTileBytes + kMisc + 1024;
};

struct WItem {
    int b, rh, blk;  // request, rank * Hkv + KV head, block of 256 tokens; b = B at the end
};

struct WBars {
    uint64_t k_full[2], k_empty[2];
    uint64_t q_full[6], q_empty[6];  // query tiles loaded / read by the products
    uint64_t i_full[2], i_empty[2];  // the even and odd ones' log-sum-exps written / read
    uint64_t s_full[2][2], s_empty[2][2];
    uint64_t x_full[2][4];           // an item's first sum written, by tile and item
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
    int plain[2];  // all the tile's rows have a finite log-sum-exp
    WItem range[2];
};
static_assert(sizeof(WBars) <= 512, "barrier region too small");

__device__ __forceinline__ int blocks_of(const ChunkParams& p, const Request& q, int r) {
    return q.n == 0 ? 0 : (rank_share(q.L, r, p.N) + 2 * kM - 1) / (2 * kM);
}
// The items in order, and what their tiles need to know; divisions only where
// the rank or the request changes.
struct WCursor {
    Request q;
    int b, r, hkv, blk;  // b = B at the end
    int nblk, held, nq_all;
    // the current item
    int tb, j0, nq;      // first token; first new token that sees the block; query tiles from there on

    __device__ __forceinline__ void rank(const ChunkParams& p) {  // the pair (b, r) has changed
        held = q.n == 0 ? 0 : rank_share(q.L, r, p.N);
        nblk = (held + 2 * kM - 1) / (2 * kM);
    }
    __device__ __forceinline__ void item(const ChunkParams& p, int tj) {
        tb = blk * 2 * kM;
        j0 = max(0, tb * p.N + r - (q.L - q.n));
        nq = j0 == 0 ? nq_all : (q.n - j0 + tj - 1) / tj;
    }
    __device__ __forceinline__ void start(const ChunkParams& p, const WItem& x, int tj) {
        b = x.b;
        if (b >= p.B) return;
        r = x.rh / p.Hkv;
        hkv = x.rh - r * p.Hkv;
        blk = x.blk;
        q = load_request(p, b);
        nq_all = (q.n + tj - 1) / tj;
        rank(p);
        item(p, tj);
    }
    // the next item that has tokens
    __device__ __forceinline__ void next(const ChunkParams& p, int tj) {
        if (++blk >= nblk) {
            blk = 0;
            if (++hkv >= p.Hkv) {
                hkv = 0;
                do {
                    if (++r >= p.N || held == 0) {  // a rank that holds nothing: nor do the later ones
                        r = 0;
                        do {
                            if (++b >= p.B) return;
                            q = load_request(p, b);
                        } while (q.n == 0 || q.L == 0);
                        nq_all = (q.n + tj - 1) / tj;
                    }
                    rank(p);
                } while (nblk == 0);
            }
        }
        item(p, tj);
    }
    __device__ __forceinline__ bool before(const ChunkParams& p, const WItem& end) const {
        return b < p.B && !(b == end.b && r * p.Hkv + hkv == end.rh && blk == end.blk);
    }
};

// The work of one KV head of a (request, rank): a block costs two (its keys and
// its sums) and one per query tile.  Blocks before `full` meet all nq of them;
// after that block k meets ceil((x - k m) / tj), m tokens of the request a block.
struct WWork {
    int nblk, full, nq;
    int64_t x, m, tj;
};
__device__ WWork head_wwork(const ChunkParams& p, int64_t pair, int tj) {
    WWork w;
    const Request q = load_request(p, (int)(pair / p.N));
    const int r = (int)(pair % p.N);
    w.nblk = blocks_of(p, q, r);
    w.nq = (q.n + tj - 1) / tj;
    w.m = (int64_t)2 * kM * p.N;
    w.tj = tj;
    w.x = (int64_t)q.L - r;
    // block k starts at the request's token k m + r: old, or the first new one, while that is <= L - n
    const int64_t old = (int64_t)q.L - q.n - r;
    w.full = old < 0 ? 0 : (int)min(old / w.m + 1, (int64_t)w.nblk);
    return w;
}
__device__ int64_t wwork_before(const WWork& w, int k) {
    const int f = min(k, w.full);
    int64_t c = (int64_t)f * w.nq + 2 * (int64_t)k;
    const int rest = k - f;  // blocks w.full .. k - 1, from the last one back: ceil((x - (k - 1) m) / tj) and up
    if (rest > 0) c += floor_sum(rest, w.tj, w.m, w.x - (int64_t)(k - 1) * w.m + w.tj - 1);
    return c;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsW, 1)
    chunk_weights_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                            const ChunkParams p) {
    using W = WShape<D>;
    constexpr int kTileBytes = W::kTileBytes, kQSlots = W::kQSlots, NCH = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* qring = smem + 4 * kTileBytes;
    float* lse_s = reinterpret_cast<float*>(qring + kQSlots * kTileBytes);
    WBars* bar = reinterpret_cast<WBars*>(lse_s + 2 * kM);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tj = kM / p.gq;  // new tokens of a query tile

    // ------------------------------------------------ this CTA's range of items
    {
        int64_t* upto = reinterpret_cast<int64_t*>(smem);  // the key buffers are not in use yet
        const int64_t npairs = (int64_t)p.B * p.N;
        const int64_t per = (npairs + kThreadsW - 1) / kThreadsW;
        int64_t sum = 0;
        for (int64_t i = tid * per; i < min((tid + 1) * per, npairs); ++i) {
            const WWork w = head_wwork(p, i, tj);
            sum += wwork_before(w, w.nblk) * p.Hkv;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(kAllLanes, sum, o);
            if (lane >= o) sum += x;
        }
        if (lane == 31) upto[kThreadsW + warp] = sum;
        __syncthreads();
        for (int w = 0; w < warp; ++w) sum += upto[kThreadsW + w];
        upto[tid] = sum;
        __syncthreads();
        const int64_t total = upto[kThreadsW - 1];
        if (lane == 0 && warp < 2) {  // the first item that starts at or after this CTA's (the next one's) share
            WItem x = {p.B, 0, 0};
            const int c = blockIdx.x + warp;
            const int64_t at = (int64_t)((double)total * c / gridDim.x);
            if (c < (int)gridDim.x && at < total) {
                int lo = 0, hi = kThreadsW - 1;
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (upto[mid] > at) hi = mid;
                    else lo = mid + 1;
                }
                int64_t rem = at - (lo ? upto[lo - 1] : 0);
                int64_t pair = lo * per;
                WWork w = head_wwork(p, pair, tj);
                int64_t head = wwork_before(w, w.nblk);
                while (rem >= head * p.Hkv) {
                    rem -= head * p.Hkv;
                    w = head_wwork(p, ++pair, tj);
                    head = wwork_before(w, w.nblk);
                }
                const int hkv = (int)(rem / head);
                rem %= head;
                int k0 = 0, k1 = w.nblk;
                while (k0 < k1) {
                    const int mid = (k0 + k1) >> 1;
                    if (wwork_before(w, mid) >= rem) k1 = mid;
                    else k0 = mid + 1;
                }
                x = {(int)(pair / p.N), (int)(pair % p.N) * p.Hkv + hkv, k0};
                if (k0 >= w.nblk) {
                    WCursor z;
                    x.blk = w.nblk - 1;
                    z.start(p, x, tj);
                    z.next(p, tj);
                    x = {z.b, z.r * p.Hkv + z.hkv, z.blk};
                    if (z.b >= p.B) x = {p.B, 0, 0};
                }
            }
            bar->range[warp] = x;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&bar->k_full[s], 1);
            mbar_init(&bar->k_empty[s], 1);
            mbar_init(&bar->i_full[s], 1);
            mbar_init(&bar->i_empty[s], 8);
            for (int i = 0; i < 4; ++i) mbar_init(&bar->x_full[s][i], 4);
            for (int u = 0; u < 2; ++u) {
                mbar_init(&bar->s_full[u][s], 1);
                mbar_init(&bar->s_empty[u][s], 4);
            }
        }
        for (int s = 0; s < kQSlots; ++s) {
            mbar_init(&bar->q_full[s], 1);
            mbar_init(&bar->q_empty[s], 1);
        }
        mbar_init(&bar->mma_done, 1);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 17) {
        tmem_alloc(&bar->tmem_base, 512);
        tmem_relinquish();
    }
    if (warp == 16 && lane == 0) {
        tma_prefetch_map(&qmap);
        tma_prefetch_map(&kmap);
    }
    fence_proxy_async_smem();  // the range's scratch is overwritten by copies
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    volatile int* abort = &bar->abort;
    int* status = &g_weights_status;
    const WItem end = bar->range[1];
    WCursor g;
    g.start(p, bar->range[0], tj);
    auto more = [&]() { return g.before(p, end); };
    bool issued_any = false;

    if (warp == 16) {
        // ---------------------------------------------------------------- TMA
        const int pb = min(1 << p.page_shift, kM);
        int it = 0, qc = 0;
        bool ok = !p.stall_loads;
        for (; ok && more(); g.next(p, tj), ++it) {
            const int kb = it & 1;
            const int tokens = min(2 * kM, g.held - g.tb);
            const int nseg = (tokens + pb - 1) / pb;  // at most 32: pages of 8 and up
            int pg = 0;
            if (lane < nseg) {  // entries of tokens that exist only
                pg = __ldg(p.bt + (int64_t)g.r * p.bt_sn + (int64_t)g.b * p.bt_sb + ((g.tb + lane * pb) >> p.page_shift));
                if ((unsigned)pg >= (unsigned)p.num_pages) pg = p.num_pages;  // reads zeros
            }
            int go = 1;
            if (lane == 0) {
                if (it >= 2) go = mbar_wait(&bar->k_empty[kb], ((it >> 1) - 1) & 1, status, DCP_ERR_TIMEOUT, abort);
                if (go) mbar_arrive_expect_tx(&bar->k_full[kb], (uint32_t)(NCH * nseg * pb * 128));
            }
            if (!__shfl_sync(kAllLanes, go, 0)) break;
            if (lane < nseg) {
                const int row = lane * pb;  // token of the block: tile row / 128
                uint8_t* dst = smem + (2 * kb + row / kM) * kTileBytes + (row % kM) * 128;
                const int slot = (g.tb + row) & ((1 << p.page_shift) - 1);
#pragma unroll
                for (int c = 0; c < NCH; ++c)
                    tma_load_5d(dst + c * kChunkB, &kmap, &bar->k_full[kb], 64 * c, g.hkv, slot, pg, g.r);
            }
            __syncwarp();
            if (lane == 0) {
                for (int k = 0; k < g.nq; ++k, ++qc) {
                    const int s = qc % kQSlots;
                    if (qc >= kQSlots &&
                        !mbar_wait(&bar->q_empty[s], (qc / kQSlots - 1) & 1, status, DCP_ERR_TIMEOUT, abort)) {
                        go = 0;
                        break;
                    }
                    // whole boxes, also past the request's last row (a smaller box for
                    // few new tokens gained nothing: 98 us either way at 64 single ones)
                    mbar_arrive_expect_tx(&bar->q_full[s], (uint32_t)(NCH * tj * p.gq * 128));
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
                        tma_load_3d(qring + s * kTileBytes + c * kChunkB, &qmap, &bar->q_full[s], 64 * c, g.hkv * p.gq,
                                    g.q.start + g.j0 + k * tj);
                }
            }
            qc = __shfl_sync(kAllLanes, qc, 0);
            if (!__shfl_sync(kAllLanes, go, 0)) break;
        }
        // copies still in flight (only after an abort) land before the CTA ends
        if (lane == 0 && *abort) {
            const uint64_t t = global_timer_ns();
            auto land = [&](uint64_t* b, int parity) {
                while (!mbar_try_wait(b, parity & 1) && global_timer_ns() - t < kWaitLimitNs) {
                }
            };
            for (int i = max(0, it - 1); i <= it; ++i) land(&bar->k_full[i & 1], i >> 1);
            for (int i = max(0, qc - kQSlots); i < qc; ++i) land(&bar->q_full[i % kQSlots], i / kQSlots);
        }
    } else if (warp == 17) {
        // ---------------------------------------------------------------- MMA
        // the whole warp runs along, its leader issues
        constexpr bool kBf16 = !std::is_same<T, __half>::value;
        const uint32_t tm = __shfl_sync(kAllLanes, tmem, 0);
        const uint32_t ka = __shfl_sync(kAllLanes, smem_u32(smem), 0);
        const uint32_t qa = ka + 4 * kTileBytes;
        auto wait = [&](uint64_t* b, int parity) -> bool {
            return __all_sync(kAllLanes, mbar_wait(b, parity & 1, status, DCP_ERR_TIMEOUT, abort));
        };
        int it = 0, qc = 0;
        unsigned used = 0u;  // phase of s_empty by tile and buffer (a barrier's phase before its first counts as done)
        bool ok = true;
        for (; ok && more(); g.next(p, tj), ++it) {
            const int nq = __shfl_sync(kAllLanes, g.nq, 0);
            const int rows = __shfl_sync(kAllLanes, (g.q.n - g.j0) * p.gq, 0);
            const int two = __shfl_sync(kAllLanes, g.held - g.tb > kM ? 1 : 0, 0);
            const int kb = it & 1;
            if (!(ok = wait(&bar->k_full[kb], it >> 1))) break;
            for (int k = 0; k < nq; ++k, ++qc) {
                const int s = qc % kQSlots;
                const int cols = min(tj * p.gq, rows - k * tj * p.gq);
                const uint32_t idesc = idesc_f16(kM, (cols + 15) & ~15, kBf16, 0, 0);
                if (!(ok = wait(&bar->q_full[s], qc / kQSlots))) break;
                const int buf = qc & 1;
                for (int u = 0; u < 1 + two; ++u) {
                    const unsigned bit = 1u << (2 * u + buf);
                    if (!(ok = wait(&bar->s_empty[u][buf], used & bit ? 0 : 1))) break;
                    used ^= bit;
                    tc_fence_after();
                    const uint64_t da = smem_desc(ka + (2 * kb + u) * kTileBytes, 16, 1024, kSwizzle128B);
                    const uint64_t db = smem_desc(qa + s * kTileBytes, 16, 1024, kSwizzle128B);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c)  // 64 elements of D a time: 16 are 32 bytes of a swizzled row
                        mma_ss4_warp<2, 2>(tm + 256 * u + kM * buf, (uint32_t)da + c * (kChunkB >> 4),
                                           (uint32_t)(da >> 32), (uint32_t)db + c * (kChunkB >> 4),
                                           (uint32_t)(db >> 32), idesc, c > 0);
                    mma_commit_warp(&bar->s_full[u][buf]);
                    issued_any = true;
                }
                if (!ok) break;
                mma_commit_warp(&bar->q_empty[s]);
            }
            if (ok) mma_commit_warp(&bar->k_empty[kb]);
        }
        if (issued_any) mma_commit_warp(&bar->mma_done);
    } else if (warp >= 18) {
        // ------------------------- log-sum-exps of the even (warp 18) and odd tiles' rows
        const int h = warp - 18;
        int qc = 0;
        bool ok = true;
        for (; ok && more(); g.next(p, tj)) {
            for (int k = 0; k < g.nq; ++k, ++qc) {
                if ((qc & 1) != h) continue;
                const int row0 = (g.j0 + k * tj) * p.gq, cols = min(tj * p.gq, g.q.n * p.gq - row0);
                float l[4];
                bool fin = true;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = 4 * lane + e;
                    l[e] = INFINITY;  // of no row, or of one that adds nothing
                    if (c < cols) {
                        const int t = c / p.gq;
                        float v = p.lse[(int64_t)(g.q.start + g.j0 + k * tj + t) * p.l_st +
                                        (int64_t)(g.hkv * p.gq + c - t * p.gq) * p.l_sh];
                        if (!p.base2) v *= kLog2e;
                        if (isfinite(v)) l[e] = v;
                        else fin = false;
                    }
                }
                if (qc >= 2 &&
                    !(ok = __all_sync(kAllLanes, mbar_wait(&bar->i_empty[h], ((qc >> 1) - 1) & 1, status,
                                                           DCP_ERR_TIMEOUT, abort))))
                    break;
                *reinterpret_cast<float4*>(lse_s + h * kM + 4 * lane) = make_float4(-l[0], -l[1], -l[2], -l[3]);
                fin = __all_sync(kAllLanes, fin);
                if (lane == 0) bar->plain[h] = fin;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->i_full[h]);
            }
        }
    } else {
        // --------------------------------------------------------------- sums
        const int u = (warp >> 2) & 1, buf = warp >> 3, m = tid & 127;
        const uint32_t tS = tmem + 256 * u + kM * buf + ((uint32_t)(32 * (warp & 3)) << 16);
        const float qscale = p.sm_scale * kLog2e;
        const Pair qs2 = pack2f(qscale, qscale);
        const float* nl = lse_s + buf * kM;  // negated log-sum-exps
        auto wait = [&](uint64_t* b, int parity) -> bool {
            return __all_sync(kAllLanes, mbar_wait(b, parity & 1, status, DCP_ERR_TIMEOUT, abort));
        };
        int qc = 0, sn = 0, xn = 0;
        bool ok = true;
        for (; ok && more(); g.next(p, tj)) {
            const int tok = g.tb + kM * u + m;
            const bool active = g.tb + kM * u < g.held;
            const int skip = (buf - qc) & 1;         // the item's first tile of this buffer
            const bool lead = skip == 0;             // whose warps write first
            qc += g.nq;
            if (skip >= g.nq) continue;              // an item of one tile: the other warps'
            float* a = p.acc + (int64_t)g.r * p.a_sn + (int64_t)g.b * p.a_sb + (int64_t)g.hkv * p.a_sh + tok;
            const float before = lead && tok < g.held && tok * p.N + g.r < g.q.L - g.q.n ? *a : 0.f;
            // new token j sees this thread's token when L - n + j >= tok N + r
            const int from = tok * p.N + g.r - (g.q.L - g.q.n);
            const int all = (min(g.held, g.tb + kM * (u + 1)) - 1) * p.N + g.r - (g.q.L - g.q.n);  // and the whole tile
            float total = 0.f;
            for (int k = skip; k < g.nq; k += 2) {
                if (!(ok = wait(&bar->i_full[buf], (qc - g.nq + k) >> 1))) break;
                if (active) {
                    if (!(ok = wait(&bar->s_full[u][buf], sn))) break;
                    ++sn;
                    tc_fence_after();
                    const int j = g.j0 + k * tj;
                    const int cols = min(tj, g.q.n - j) * p.gq;
                    // every row has a finite log-sum-exp and sees every token of the tile
                    const bool plain = *(volatile int*)&bar->plain[buf] != 0 && j >= all;
                    // the first column that sees this token, 0 when all do: `from` falls to minus the
                    // request's length, which times the group passes 32 bits
                    const int first = max(from - j, 0) * p.gq;
                    Pair acc[2] = {0ull, 0ull};
                    float part[2] = {0.f, 0.f};
                    for (int c0 = 0; c0 < cols; c0 += 32) {
                        uint32_t v[32];
                        tmem_ld32<0>(tS + c0, v);
                        tmem_wait_ld();
                        pin(v);
                        if (plain && c0 + 32 <= cols) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(nl + c0 + e);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float2 y =
                                        unpack2(fma2(pack2(v[e + 2 * h], v[e + 2 * h + 1]), qs2, h ? l.y : l.x));
                                    add2(acc[h], pack2f(exp2_fast(y.x), exp2_fast(y.y)));
                                }
                            }
                        } else {
                            // columns of no row, and of rows that add nothing, hold -infinity
                            // here; their scores may be anything
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 l4 = *reinterpret_cast<const float4*>(nl + c0 + e);
                                const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    const float w = exp2_fast(fmaf(__uint_as_float(v[e + h]), qscale, l[h]));
                                    part[h & 1] += c0 + e + h >= first && l[h] != -INFINITY ? w : 0.f;
                                }
                            }
                        }
                    }
                    const float2 a0 = unpack2(acc[0]), a1 = unpack2(acc[1]);
                    total += ((a0.x + a0.y) + (a1.x + a1.y)) + (part[0] + part[1]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->s_empty[u][buf]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar->i_empty[buf]);
            }
            // the sums of an item's even and odd tiles, in a fixed order.  A tile without
            // tokens has none to exchange, and its warps wait for no scores: they would not
            // be held back.  In the others the writer is at most two exchanges ahead of the
            // reader: of the items after the reader's, each has a tile of the reader's score
            // buffer, the first of them fills it, and the next item's products stop there.
            if (g.nq > 1) {
                if (!active) continue;
                if (lead) {
                    if (ok && tok < g.held) __stcg(a, before + total);
                    __threadfence();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar->x_full[u][xn & 3]);
                } else {
                    ok = ok && wait(&bar->x_full[u][xn & 3], xn >> 2);
                    __threadfence();
                    if (ok && tok < g.held) __stcg(a, __ldcg(a) + total);
                }
                ++xn;
            } else if (ok && tok < g.held) {
                *a = before + total;
            }
        }
    }

    // --------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        if (lane == 0 && issued_any) {
            // every MMA this CTA issued has completed before its tensor memory goes
            const uint64_t t = global_timer_ns();
            while (!mbar_try_wait(&bar->mma_done, 0) && global_timer_ns() - t < kWaitLimitNs) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int D>
cudaError_t launch_weights_tc(const ChunkParams& p, const CUtensorMap (&maps)[2], cudaStream_t stream) {
    const void* k = (const void*)chunk_weights_tc_kernel<T, D>;
    // the shared-memory opt-in is a per-device function attribute
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, WShape<D>::kSmem);
    if (e != cudaSuccess) return e;
    chunk_weights_tc_kernel<T, D>
        <<<device_sm_count(), kThreadsW, WShape<D>::kSmem, stream>>>(maps[0], maps[1], p);
    return cudaGetLastError();
}

}  // namespace

bool launch_chunk_weights_tc(const ChunkParams& p, int dtype, cudaStream_t stream, cudaError_t* err) {
    // boxes hold whole 8-row swizzle atoms.  Where both kernels can run this one takes
    // 97 against 147 us (64 single tokens over 8192), 74 against 178 (ragged, 12 heads a
    // group), 277 against 1412 (2048 new), 20 against 26 (32 ragged requests of up to 40
    // over 500), 11.8 against 12.2 (8 of up to 20 over 300).  It loses by its set-up where
    // there is little to do: 8.7 against 4.3 (one token over 64), 12.7 against 5.7 (64
    // single tokens over 128), 26 against 13 (256 requests, 2 over 100).  The lengths
    // that tell these apart are on the device; max_seq_len bounds them only
    if ((p.D != 64 && p.D != 128) || p.page_shift < 3) return false;
    const EncodeTiledFn enc = tensor_map_encoder();
    if (!enc) return false;
    const CUtensorMapDataType dt = dtype == DCP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    // a dimension of extent 1 is never stepped over: give it a nominal stride
    auto stride = [](int64_t extent, int64_t bytes) -> cuuint64_t { return (cuuint64_t)(extent > 1 ? bytes : 256); };
    CUtensorMap maps[2];
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
    {
        const int64_t rows = (int64_t)1 << p.page_shift;
        const cuuint64_t dims[5] = {(cuuint64_t)p.D, (cuuint64_t)p.Hkv, (cuuint64_t)rows, (cuuint64_t)p.num_pages,
                                    (cuuint64_t)p.N};
        const cuuint64_t strides[4] = {stride(p.Hkv, p.k_sh), stride(rows, p.k_st), stride(p.num_pages, p.k_sp),
                                       stride(p.N, p.k_sn)};
        const cuuint32_t box[5] = {64, 1, (cuuint32_t)(rows < kM ? rows : kM), 1, 1};
        if (enc(&maps[1], dt, 5, p.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
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
        *err = dtype == DCP_F16 ? launch_weights_tc<__half, 128>(q, maps, stream)
                                : launch_weights_tc<__nv_bfloat16, 128>(q, maps, stream);
    else
        *err = dtype == DCP_F16 ? launch_weights_tc<__half, 64>(q, maps, stream)
                                : launch_weights_tc<__nv_bfloat16, 64>(q, maps, stream);
    return true;
}

int chunk_weights_tc_status(bool clear) {
    int s = 0;
    if (cudaMemcpyFromSymbol(&s, g_weights_status, sizeof(int)) != cudaSuccess) return -1;
    if (clear && s) {
        const int zero = 0;
        if (cudaMemcpyToSymbol(g_weights_status, &zero, sizeof(int)) != cudaSuccess) return -1;
    }
    return s;
}

}  // namespace dcp
