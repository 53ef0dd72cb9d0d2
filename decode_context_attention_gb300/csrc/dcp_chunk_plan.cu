// dcp_chunk_plan.cu -- the split of a ragged batch's chunk attention over the
// CTAs, and the merge of the results of the items that the split cuts.
//
// The plan is one CTA of 1024 threads: it reads 12 bytes per request and writes
// 16 per range, so its time is that of a few dependent loads.  The tiles that a
// block of new tokens sees are floor((a qt + b) / M) in its index qt, so a
// request's work up to any block is a sum of floors, which Euclid's steps
// give without a loop over the blocks: a thread sums a (request, rank) pair at
// once, and a thread per range finds its start by bisection.  (A warp per pair
// and boundary, looping over blocks: 24 us for 32 requests of 16384 tokens on 4
// ranks, 61 us for one of 4096 new tokens.)
// The merge reads and writes what the cuts left, at most two partial blocks per
// CTA: a warp takes four rows, all their parts in flight.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kItemCost = 2;  // fixed part of an item's work, in tiles
constexpr int kMinPart = 4;   // a cut leaves at least this many tiles on both sides
constexpr int kPlanThreads = 1024;
constexpr unsigned kAll = 0xffffffffu;

// The work of one KV head of a (request, rank), by blocks of new tokens.
struct HeadWork {
    int nq;       // blocks
    int last;     // tiles of the last one
    int q0;       // blocks that see nothing because the request has more new tokens than tokens
    int64_t a, b, m;
};
__device__ HeadWork head_work(const ChunkParams& p, int pair, int tpi, int tt) {
    HeadWork w;
    const int r = pair % p.N;
    const Request q = load_request(p, pair / p.N);
    w.nq = (q.n + tpi - 1) / tpi;
    w.last = (rank_share(q.L, r, p.N) + tt - 1) / tt;  // its last row is the request's last token
    w.q0 = 0;
    w.m = (int64_t)p.N * tt;
    if (p.causal) {
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
__device__ int64_t work_before(const HeadWork& w, int q) {
    const int k = min(q, w.nq - 1) - w.q0;
    int64_t c = (int64_t)q * kItemCost;
    if (k > 0) c += floor_sum(k, w.m, w.a, w.b);
    if (q >= w.nq && w.nq > 0) c += w.last;
    return c;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p, int tpi, int tt, int ctas,
                                                                  ChunkPos* pos) {
    __shared__ int64_t upto[kPlanThreads];  // work up to and with a thread's pairs
    __shared__ int64_t warp_sum[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t npairs = (int64_t)p.B * p.N;
    const int64_t per = (npairs + kPlanThreads - 1) / kPlanThreads;
    int64_t sum = 0;
    for (int64_t i = tid * per; i < min((tid + 1) * per, npairs); ++i) {
        const HeadWork w = head_work(p, (int)i, tpi, tt);
        sum += work_before(w, w.nq) * p.Hkv;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    upto[tid] = before + sum;
    __syncthreads();
    const int64_t total = upto[kPlanThreads - 1];
    for (int c = tid; c <= ctas; c += kPlanThreads) {
        ChunkPos x = {p.B, 0, 0, 0};
        const int64_t at = (int64_t)((double)total * c / ctas);  // exact below 2^53 / ctas, monotone above
        if (c < ctas && at < total) {
            int lo = 0, hi = kPlanThreads - 1;  // the first thread whose pairs pass `at`
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (upto[mid] > at) hi = mid;
                else lo = mid + 1;
            }
            int64_t rem = at - (lo ? upto[lo - 1] : 0);
            int64_t pair = lo * per;
            HeadWork w = head_work(p, (int)pair, tpi, tt);
            int64_t head = work_before(w, w.nq);
            while (rem >= head * p.Hkv) {  // `at` lies in one of this thread's pairs
                rem -= head * p.Hkv;
                w = head_work(p, (int)++pair, tpi, tt);
                head = work_before(w, w.nq);
            }
            const int b = (int)(pair / p.N), r = (int)(pair % p.N);
            const int hkv = (int)(rem / head);
            rem %= head;
            int q0 = 0, q1 = w.nq - 1;  // the last block whose work starts at or before rem
            while (q0 < q1) {
                const int mid = (q0 + q1 + 1) >> 1;
                if (work_before(w, mid) <= rem) q0 = mid;
                else q1 = mid - 1;
            }
            const int64_t begin = work_before(w, q0);
            const int n = (int)(work_before(w, q0 + 1) - begin) - kItemCost, off = (int)(rem - begin);
            x = {b, r * p.Hkv + hkv, q0, max(off - kItemCost, 0)};
            // a cut near an end of its item, or into a short one, moves to the nearer end
            if (2 * off < n + kItemCost) {
                if (x.tile < kMinPart || n < 2 * kMinPart) x.tile = 0;
            } else if (n - x.tile < kMinPart || n < 2 * kMinPart) {
                x = next_item(p, x, tpi);
            }
        }
        pos[c] = x;
    }
}

// CTA c0 joins the item whose first part is the last one of range c0: slot
// 2 c0 (the range's first item) or 2 c0 + 1, then slot 2 c of every range c up
// to the one that ends the item.
constexpr int kMergeRows = 4;  // rows of a warp

template <typename T, int D>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p, const ChunkPartials ws, int tpi,
                                                          int rows) {
    constexpr int NV = (D + 127) / 128;  // 16-byte vectors of a lane
    const int c0 = blockIdx.x;
    const ChunkPos x = ws.pos[c0 + 1], y = ws.pos[c0];
    if (x.b >= p.B || x.tile == 0) return;
    if (same_item(x, y) && y.tile > 0) return;  // an earlier range holds the item's first part
    const Request q = load_request(p, x.b);
    const int r = x.rh / p.Hkv, hkv = x.rh % p.Hkv;
    const int j0 = x.qt * tpi;
    const int nrows = min(tpi, q.n - j0) * p.gq;
    const int row0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kMergeRows, lane = threadIdx.x & 31;
    if (row0 >= nrows) return;
    const int s0 = 2 * c0 + (same_item(x, y) ? 0 : 1);
    int c1 = c0 + 1;
    for (ChunkPos z; c1 + 1 < (int)gridDim.x; ++c1) {
        z = ws.pos[c1 + 1];
        if (!same_item(z, x) || z.tile == 0) break;
    }
    // a range that lies empty inside the item left nothing
    auto empty = [&](int c) { return same_item(ws.pos[c], ws.pos[c + 1]) && ws.pos[c].tile == ws.pos[c + 1].tile; };
    float mx[kMergeRows], sum[kMergeRows];
    float4 acc[kMergeRows][NV];
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k) {
        mx[k] = -INFINITY;
        sum[k] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) acc[k][v] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int c = c0; c <= c1; ++c) {
        if (c != c0 && empty(c)) continue;
        const int64_t at = (int64_t)(c == c0 ? s0 : 2 * c) * rows + row0;
#pragma unroll
        for (int k = 0; k < kMergeRows; ++k)
            if (row0 + k < nrows) mx[k] = fmaxf(mx[k], ws.lse[at + k]);
    }
    for (int c = c0; c <= c1; ++c) {
        if (c != c0 && empty(c)) continue;
        const int64_t at = (int64_t)(c == c0 ? s0 : 2 * c) * rows + row0;
        float w[kMergeRows];
        float4 o[kMergeRows][NV];
#pragma unroll
        for (int k = 0; k < kMergeRows; ++k) {
            w[k] = row0 + k < nrows ? ws.lse[at + k] : -INFINITY;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (row0 + k < nrows && 4 * lane + 128 * v < D)
                    o[k][v] = *reinterpret_cast<const float4*>(ws.o + (at + k) * D + 4 * lane + 128 * v);
                else o[k][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kMergeRows; ++k) {
            if (w[k] == -INFINITY) continue;
            w[k] = exp2f(w[k] - mx[k]);  // mx is finite, infinite or NaN with w: as the formula has it
            sum[k] += w[k];
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                acc[k][v].x = fmaf(w[k], o[k][v].x, acc[k][v].x);
                acc[k][v].y = fmaf(w[k], o[k][v].y, acc[k][v].y);
                acc[k][v].z = fmaf(w[k], o[k][v].z, acc[k][v].z);
                acc[k][v].w = fmaf(w[k], o[k][v].w, acc[k][v].w);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kMergeRows; ++k) {
        const int row = row0 + k;
        if (row >= nrows) break;
        const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
        const int t = q.start + j0 + row / p.gq, h = hkv * p.gq + row % p.gq;
        unsigned char* out = p.o + (int64_t)r * p.o_sn + (int64_t)t * p.o_st + (int64_t)h * p.o_sh;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (4 * lane + 128 * v < D) {
                const float4 a = acc[k][v];
                *reinterpret_cast<uint2*>(out + 2 * (4 * lane + 128 * v)) =
                    make_uint2(f32_to_pair(make_float2(a.x * inv, a.y * inv), T()),
                               f32_to_pair(make_float2(a.z * inv, a.w * inv), T()));
            }
        if (lane == 0) {
            const float lse2 = sum[k] == 0.f ? -INFINITY : mx[k] + log2f(sum[k]);
            p.lse[(int64_t)r * p.l_sn + (int64_t)t * p.l_st + (int64_t)h * p.l_sh] = p.base2 ? lse2 : lse2 * kLn2;
        }
    }
}

template <typename T>
void launch_merge(const ChunkParams& p, const ChunkPartials& ws, int tpi, int rows, dim3 grid, cudaStream_t stream) {
    switch (p.D) {
        case 64: chunk_merge_kernel<T, 64><<<grid, 256, 0, stream>>>(p, ws, tpi, rows); break;
        case 128: chunk_merge_kernel<T, 128><<<grid, 256, 0, stream>>>(p, ws, tpi, rows); break;
        default: chunk_merge_kernel<T, 256><<<grid, 256, 0, stream>>>(p, ws, tpi, rows); break;
    }
}

constexpr size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

size_t chunk_partials_bytes(int ctas, int rows, int D) {
    return align256((size_t)(ctas + 1) * sizeof(ChunkPos)) + align256((size_t)2 * ctas * rows * D * 4) +
           align256((size_t)2 * ctas * rows * 4);
}
ChunkPartials chunk_partials_in(unsigned char* ws, int ctas, int rows, int D) {
    ChunkPartials x;
    x.pos = reinterpret_cast<ChunkPos*>(ws);
    x.o = reinterpret_cast<float*>(ws + align256((size_t)(ctas + 1) * sizeof(ChunkPos)));
    x.lse = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(x.o) + align256((size_t)2 * ctas * rows * D * 4));
    return x;
}

cudaError_t launch_chunk_plan(const ChunkParams& p, const ChunkPartials& ws, int tpi, int tt, int ctas,
                              cudaStream_t stream) {
    chunk_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, tpi, tt, ctas, ws.pos);
    return cudaGetLastError();
}
cudaError_t launch_chunk_merge(const ChunkParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                               cudaStream_t stream) {
    const dim3 grid(ctas, (tpi * p.gq + 8 * kMergeRows - 1) / (8 * kMergeRows));
    if (dtype == DCP_F16) launch_merge<__half>(p, ws, tpi, rows, grid, stream);
    else launch_merge<__nv_bfloat16>(p, ws, tpi, rows, grid, stream);
    return cudaGetLastError();
}

}  // namespace dcp
