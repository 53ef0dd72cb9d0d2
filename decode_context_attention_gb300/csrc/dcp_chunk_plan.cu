// dcp_chunk_plan.cu -- the split of a ragged batch's chunk attention over the
// CTAs, and the merge of the results of the items that the split cuts.
//
// The plan is one CTA of 1024 threads; it reads 12 bytes per request and
// writes 16 per range.  The merge reads and writes what the cuts left, at most
// two partial blocks per CTA.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kItemCost = 2;  // fixed part of an item's work, in tiles
constexpr int kMinPart = 4;   // a cut leaves at least this many tiles in front of it
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// Work of one KV head of (request, rank), in tiles: blocks lane, lane + step, ...
__device__ int64_t head_cost(const ChunkParams& p, const Request& q, int r, int tpi, int tt, int lane, int step) {
    int64_t c = 0;
    for (int qt = lane; qt * tpi < q.n; qt += step) c += item_tiles(p, q, r, qt, tpi, tt) + kItemCost;
    return c;
}
__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
__device__ __forceinline__ int64_t warp_scan64(int64_t v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kAll, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The costs (one KV head) of 32 (request, rank) pairs, one per lane; a pair of
// many blocks is summed by the whole warp.  pair >= npairs costs nothing.
__device__ int64_t pair_costs(const ChunkParams& p, int pair, int npairs, int tpi, int tt, int lane) {
    Request q = {0, 0, 0};
    int r = 0;
    if (pair < npairs) {
        q = load_request(p, pair / p.N);
        r = pair % p.N;
    }
    const bool many = q.n > 8 * tpi;
    int64_t c = many ? 0 : head_cost(p, q, r, tpi, tt, 0, 1);
    for (unsigned m = __ballot_sync(kAll, many); m; m &= m - 1) {
        const int src = __ffs(m) - 1;
        Request x;
        x.start = 0;
        x.n = __shfl_sync(kAll, q.n, src);
        x.L = __shfl_sync(kAll, q.L, src);
        const int xr = __shfl_sync(kAll, r, src);
        const int64_t s = warp_sum64(head_cost(p, x, xr, tpi, tt, lane, 32));
        if (lane == src) c = s;
    }
    return c;
}

// Where each of the `ctas` ranges starts; pos[ctas] is the end.  Two sweeps over
// the (request, rank) pairs, the first for the total, the second by one warp
// per range boundary.
__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const ChunkParams p, int tpi, int tt, int ctas,
                                                                  ChunkPos* pos) {
    __shared__ int64_t before[kPlanWarps + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int npairs = p.B * p.N;
    const int per = ((npairs + kPlanWarps - 1) / kPlanWarps + 31) & ~31;
    const int64_t w0 = (int64_t)warp * per;
    const int lo = (int)min(w0, (int64_t)npairs), hi = (int)min(w0 + per, (int64_t)npairs);
    int64_t sum = 0;
    for (int i = lo; i < hi; i += 32) sum += pair_costs(p, i + lane < hi ? i + lane : npairs, npairs, tpi, tt, lane);
    sum = warp_sum64(sum) * p.Hkv;
    if (lane == 0) before[warp + 1] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        before[0] = 0;
        for (int w = 0; w < kPlanWarps; ++w) before[w + 1] += before[w];
    }
    __syncthreads();
    const int64_t total = before[kPlanWarps];
    for (int c = warp; c <= ctas; c += kPlanWarps) {
        ChunkPos x = {p.B, 0, 0, 0};
        const int64_t at = (int64_t)((double)total * c / ctas);  // exact below 2^53 / ctas, monotone above
        if (c < ctas && at < total) {
            int w = 0;
            while (before[w + 1] <= at) ++w;
            int64_t rem = at - before[w];
            const int stop = (int)min((int64_t)(w + 1) * per, (int64_t)npairs);
            for (int i = w * per; i < stop; i += 32) {
                const int64_t mine = pair_costs(p, i + lane < stop ? i + lane : npairs, npairs, tpi, tt, lane);
                const int64_t upto = warp_scan64(mine * p.Hkv, lane);
                const unsigned past = __ballot_sync(kAll, upto > rem);
                if (!past) {
                    rem -= __shfl_sync(kAll, upto, 31);
                    continue;
                }
                const int src = __ffs(past) - 1;
                const int64_t head = __shfl_sync(kAll, mine, src);
                rem -= __shfl_sync(kAll, upto, src) - head * p.Hkv;
                const int pair = i + src, b = pair / p.N, r = pair % p.N;
                const Request q = load_request(p, b);
                const int hkv = (int)(rem / head);
                rem %= head;
                for (int q0 = 0; q0 * tpi < q.n; q0 += 32) {  // rem < head, so an item is found
                    const int qt = q0 + lane;
                    const int tiles = qt * tpi < q.n ? item_tiles(p, q, r, qt, tpi, tt) : -kItemCost;
                    const int64_t up = warp_scan64(tiles + kItemCost, lane);
                    const unsigned hit = __ballot_sync(kAll, up > rem);
                    if (!hit) {
                        rem -= __shfl_sync(kAll, up, 31);
                        continue;
                    }
                    const int k = __ffs(hit) - 1;
                    const int n = __shfl_sync(kAll, tiles, k);
                    const int off = (int)(rem - (__shfl_sync(kAll, up, k) - n - kItemCost));
                    x = {b, r * p.Hkv + hkv, q0 + k, max(off - kItemCost, 0)};
                    // a cut near an end of its item, or into a short one, moves to the nearer end
                    if (2 * off < n + kItemCost) {
                        if (x.tile < kMinPart || n < 2 * kMinPart) x.tile = 0;
                    } else if (n - x.tile < kMinPart || n < 2 * kMinPart) {
                        x = next_item(p, x, tpi);
                    }
                    break;
                }
                break;
            }
        }
        if (lane == 0) pos[c] = x;
    }
}

// CTA c0 joins the item whose first part is the last one of range c0: slot
// 2 c0 (the range's first item) or 2 c0 + 1, then slot 2 c of every range c up
// to the one that ends the item.  One warp per row.
template <typename T>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const ChunkParams p, const ChunkPartials ws, int tpi,
                                                          int rows) {
    const int c0 = blockIdx.x;
    const ChunkPos x = ws.pos[c0 + 1];
    if (x.b >= p.B || x.tile == 0) return;
    const ChunkPos y = ws.pos[c0];
    if (same_item(x, y) && y.tile > 0) return;  // an earlier range holds the item's first part
    const Request q = load_request(p, x.b);
    const int r = x.rh / p.Hkv, hkv = x.rh % p.Hkv;
    const int j0 = x.qt * tpi;
    const int nrows = min(tpi, q.n - j0) * p.gq;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= nrows) return;
    const int s0 = 2 * c0 + (same_item(x, y) ? 0 : 1);
    int c1 = c0 + 1;
    while (c1 + 1 < (int)gridDim.x && same_item(ws.pos[c1 + 1], x) && ws.pos[c1 + 1].tile > 0) ++c1;
    auto empty = [&](int c) { return same_item(ws.pos[c], ws.pos[c + 1]) && ws.pos[c].tile == ws.pos[c + 1].tile; };
    float mx = ws.lse[(int64_t)s0 * rows + row];
    for (int c = c0 + 1; c <= c1; ++c)
        if (!empty(c)) mx = fmaxf(mx, ws.lse[(int64_t)(2 * c) * rows + row]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float acc[8], sum = 0.f;  // elements lane + 32 k of the row (D <= 256)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    for (int c = c0; c <= c1; ++c) {
        if (c != c0 && empty(c)) continue;
        const int s = c == c0 ? s0 : 2 * c;
        const float lse = ws.lse[(int64_t)s * rows + row];
        if (lse == -INFINITY) continue;
        const float w = exp2f(lse - base);
        sum += w;
        const float* o = ws.o + ((int64_t)s * rows + row) * p.D;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (lane + 32 * k < p.D) acc[k] = fmaf(w, o[lane + 32 * k], acc[k]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float lse2 = sum == 0.f ? -INFINITY : base + log2f(sum);
    const int t = q.start + j0 + row / p.gq, h = hkv * p.gq + row % p.gq;
    T* out = reinterpret_cast<T*>(p.o + (int64_t)r * p.o_sn + (int64_t)t * p.o_st + (int64_t)h * p.o_sh);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (lane + 32 * k < p.D) out[lane + 32 * k] = from_f32<T>(acc[k] * inv);
    if (lane == 0)
        p.lse[(int64_t)r * p.l_sn + (int64_t)t * p.l_st + (int64_t)h * p.l_sh] = p.base2 ? lse2 : lse2 * kLn2;
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
    const dim3 grid(ctas, (tpi * p.gq + 7) / 8);
    if (dtype == DCP_F16) chunk_merge_kernel<__half><<<grid, 256, 0, stream>>>(p, ws, tpi, rows);
    else chunk_merge_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(p, ws, tpi, rows);
    return cudaGetLastError();
}

}  // namespace dcp
