// dcp_chunk_merge.cu -- the merge of the partial results that the split of a ragged
// batch's chunk attention leaves, and the layout of its workspace.
//
// The merge reads and writes what the cuts left, at most two partial blocks per
// CTA: a warp takes four rows, all their parts in flight.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

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
    // two parts at a time, all their rows in flight
    for (int c = c0; c <= c1; c += 2) {
        float w[2][kMergeRows];
        float4 o[2][kMergeRows][NV];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool there = c + e <= c1 && (c + e == c0 || !empty(c + e));
            const int64_t at = (int64_t)(c + e == c0 ? s0 : 2 * (c + e)) * rows + row0;
#pragma unroll
            for (int k = 0; k < kMergeRows; ++k) {
                const bool ok = there && row0 + k < nrows;
                w[e][k] = ok ? ws.lse[at + k] : -INFINITY;
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    if (ok && 4 * lane + 128 * v < D)
                        o[e][k][v] = *reinterpret_cast<const float4*>(ws.o + (at + k) * D + 4 * lane + 128 * v);
                    else o[e][k][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int k = 0; k < kMergeRows; ++k) {
            // mx becomes finite, infinite or NaN with the parts: as the formula has it
            const float m = fmaxf(mx[k], fmaxf(w[0][k], w[1][k]));
            const float old = mx[k] == -INFINITY ? 0.f : exp2f(mx[k] - m);
            const float w0 = w[0][k] == -INFINITY ? 0.f : exp2f(w[0][k] - m);
            const float w1 = w[1][k] == -INFINITY ? 0.f : exp2f(w[1][k] - m);
            mx[k] = m;
            sum[k] = fmaf(sum[k], old, w0 + w1);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                float4& x = acc[k][v];
                const float4 &x0 = o[0][k][v], &x1 = o[1][k][v];
                x.x = fmaf(w1, x1.x, fmaf(w0, x0.x, x.x * old));
                x.y = fmaf(w1, x1.y, fmaf(w0, x0.y, x.y * old));
                x.z = fmaf(w1, x1.z, fmaf(w0, x0.z, x.z * old));
                x.w = fmaf(w1, x1.w, fmaf(w0, x0.w, x.w * old));
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
cudaError_t launch_merge(const ChunkParams& p, const ChunkPartials& ws, int tpi, int rows, dim3 grid,
                         cudaStream_t stream) {
    const void* k = p.D == 64 ? (const void*)chunk_merge_kernel<T, 64>
                              : p.D == 128 ? (const void*)chunk_merge_kernel<T, 128> : (const void*)chunk_merge_kernel<T, 256>;
    void* args[] = {const_cast<ChunkParams*>(&p), const_cast<ChunkPartials*>(&ws), &tpi, &rows};
    return cudaLaunchKernel(k, grid, dim3(256), args, 0, stream);
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

cudaError_t launch_chunk_merge(const ChunkParams& p, const ChunkPartials& ws, int tpi, int tt, int rows, int ctas,
                               int dtype, cudaStream_t stream) {
    const int64_t cap = ((int64_t)p.max_seq_len + p.N - 1) / p.N;
    if ((cap + tt - 1) / tt < 2 * kMinPart) return cudaSuccess;
    const dim3 grid(ctas, (tpi * p.gq + 8 * kMergeRows - 1) / (8 * kMergeRows));
    return dtype == DCP_F16 ? launch_merge<__half>(p, ws, tpi, rows, grid, stream)
                            : launch_merge<__nv_bfloat16>(p, ws, tpi, rows, grid, stream);
}

}  // namespace dcp
