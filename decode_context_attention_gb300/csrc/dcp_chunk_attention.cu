// dcp_chunk_attention.cu -- attention of a ragged batch's new tokens over every
// rank's paged cache: the register-tiled kernel, which takes every shape.
//
// sglang PR #34213 report, "功能与动机": the cached-extend merge joins per-rank
// partials of an extend; sglang PR #33926 report, "关键源码片段"
// (`get_dcp_lens`): rank r holds L / N tokens plus one when r < L % N, so the
// new token of global index g sees get_dcp_lens(g + 1) local tokens.
//
// Per rank, request and KV head the rows are (new token, query head of the
// group), token-major, so a block of rows shares the KV head's tiles and the
// number of visible tokens does not fall from row to row.  One pass over the
// tiles with the running maximum m and sum l of an online softmax in base 2:
//     m' = max(m, max_i s_i),  l' = l 2^(m - m') + sum_i 2^(s_i - m'),
//     O' = O 2^(m - m') + sum_i 2^(s_i - m') v_i.
//
// The kernel runs on mma.sync (m16n8k16): 64 rows a CTA, 16 a warp, tiles of 64
// tokens staged in shared memory by cp.async, two or three CTAs an SM covering one
// another's copies.  It is bound by the warp-level products' rate: 255 TFLOP/s at
// D = 128 (4096 new tokens over 32768), 224 at D = 256 (1024 over 4096, 536 us).
// 4 new tokens of 32 requests of 16384 at D = 256: 631 us, 3.4 TB/s.  The tcgen05 kernel
// takes over for D = 64 and 128, positive scales and pages of 8 tokens and more.
#include <type_traits>

#include "dcp_chunk.cuh"
#include "dcp_mma.cuh"

namespace dcp {
namespace {

constexpr int kRows = 64;  // rows of a CTA
constexpr int kTile = 64;  // tokens of a tile
constexpr int kThreadsMma = 128;

template <int D>
struct MmaShape {
    static constexpr int kPitch = D * 2 + 16;  // bytes of a staged row: 16 more keep ldmatrix free of bank conflicts
    static constexpr int kSmem = (kRows + 2 * kTile) * kPitch;
};

// The weights, at most 1, are multiplied by this for the value product: fp16's smallest
// normal is 2^-14, so weights below it would lose bits and those below 2^-25 be lost,
// while the row sum keeps them.  Beside 2^15 the same holds from 2^-29 and 2^-40 of the
// row's largest on.  A power of two, exact; O is divided by it at the end.
template <typename T>
constexpr float kWeightUnit = std::is_same<T, __half>::value ? 32768.f : 1.f;

template <typename T, int D, class Params>
__global__ void __launch_bounds__(kThreadsMma) chunk_attention_kernel(const Params p, const ChunkPartials ws,
                                                                      int tpi) {
    constexpr bool kPlanned = std::is_same<Params, PrefixParams>::value;
    if constexpr (kPlanned) {
        chain_wait();     // the plan
        chain_release();  // what follows, which reads the plan too
        if (*p.nothing) return;
    }
    constexpr int P = MmaShape<D>::kPitch;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned char* qs = smem;
    unsigned char* ks = smem + kRows * P;
    unsigned char* vs = ks + kTile * P;
    __shared__ unsigned poison[4][2];  // tokens of the item's masked tiles whose V row is not finite
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ ChunkPos range[2];
    find_range<kThreadsMma>(p, tpi, tpi, kTile, ws.pos, reinterpret_cast<int64_t*>(smem), range);
    ChunkPos x = range[0];
    const ChunkPos end = range[1];
    const ChunkPos first = x;
    const float qscale = p.sm_scale * kLog2e;

    while (x.b < p.B && !(same_item(x, end) && x.tile == end.tile)) {
        const auto q = load_request(p, x.b);
        const int r = x.rh / p.Hkv, hkv = x.rh % p.Hkv;
        const int64_t table = table_at(p, q, r, x.b);
        const int j0 = x.qt * tpi;
        const int nrows = min(tpi, q.n - j0) * p.gq;
        const int ntiles = item_tiles(p, q, r, x.qt, tpi, kTile);
        const bool cut = same_item(x, end);
        const int t0 = x.tile, t1 = cut ? end.tile : ntiles;
        const bool whole = t0 == 0 && t1 == ntiles;
        const int slot = 2 * blockIdx.x + (same_item(x, first) ? 0 : 1);
        const int lim0 = visible(p, q, j0, r);  // the fewest tokens a row of the item sees
        const int lim_last = visible(p, q, min(j0 + tpi, q.n) - 1, r);
        const int mtile = lim0 / kTile;         // tiles from here on are masked
        // rows of this thread: two of the warp's sixteen
        int lim[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = warp * 16 + (lane >> 2) + 8 * i;
            lim[i] = row < nrows ? visible(p, q, j0 + row / p.gq, r) : 0;
        }
        __syncthreads();  // the previous item is done with shared memory
        if (tid < 8) poison[tid >> 1][tid & 1] = 0u;
        for (int id = tid; id < kRows * (D / 8); id += kThreadsMma) {
            const int row = id / (D / 8), u = id % (D / 8);
            const unsigned char* src = p.q;
            const bool ok = row < nrows;
            if (ok)
                src += (int64_t)(q.start + j0 + row / p.gq) * p.q_st + (int64_t)(hkv * p.gq + row % p.gq) * p.q_sh +
                       16 * u;
            copy16(qs + row * P + 16 * u, src, ok);
        }
        copy_commit();
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        for (int t = t0; t < t1; ++t) {
            const int tb = t * kTile;
            __syncthreads();  // every warp is done with the previous tile
            for (int id = tid; id < kTile * (D / 8); id += kThreadsMma) {
                const int row = id / (D / 8), u = id % (D / 8), i = tb + row;
                const int pg = i < lim_last ? page_in(p, table, i) : -1;
                const unsigned char *ka = p.k, *va = p.v;
                if (pg >= 0) {
                    ka += k_offset(p, r, pg, i, hkv) + 16 * u;
                    va += v_offset(p, r, pg, i, hkv) + 16 * u;
                }
                copy16(ks + row * P + 16 * u, ka, pg >= 0);
                copy16(vs + row * P + 16 * u, va, pg >= 0);
            }
            copy_commit();
            copy_wait<0>();
            __syncthreads();
            const bool masked = tb + kTile > lim0;
            if (masked) {
                // a value that some rows may not see must not reach them as 0 * inf
                for (int id = tid; id < kTile * (D / 8); id += kThreadsMma) {
                    const int row = id / (D / 8), u = id % (D / 8);
                    uint4* at = reinterpret_cast<uint4*>(vs + row * P + 16 * u);
                    uint4 v = *at;
                    if (pair_nonfinite<T>(v.x) || pair_nonfinite<T>(v.y) || pair_nonfinite<T>(v.z) ||
                        pair_nonfinite<T>(v.w)) {
                        v = make_uint4(pair_finite<T>(v.x), pair_finite<T>(v.y), pair_finite<T>(v.z),
                                       pair_finite<T>(v.w));
                        *at = v;
                        atomicOr(&poison[t - mtile][row >> 5], 1u << (row & 31));
                    }
                }
                __syncthreads();
            }
            // scores: 16 rows x 64 tokens a warp
            float s[kTile / 8][4];
#pragma unroll
            for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[n][c] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                unsigned a[4];
                ldsm4(a, smem_addr(qs + (warp * 16 + (lane & 15)) * P + 32 * kk + 16 * (lane >> 4)));
#pragma unroll
                for (int n = 0; n < kTile / 16; ++n) {
                    unsigned b[4];
                    ldsm4(b, smem_addr(ks + (n * 16 + (lane & 7) + 8 * (lane >> 4)) * P + 32 * kk +
                                       16 * ((lane >> 3) & 1)));
                    mma16816<T>(s[2 * n], a, b[0], b[1]);
                    mma16816<T>(s[2 * n + 1], a, b[2], b[3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float mx = -INFINITY;
#pragma unroll
                for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float& v = s[n][2 * i + c];
                        v *= qscale;
                        if (masked && tb + n * 8 + (lane & 3) * 2 + c >= lim[i]) v = -INFINITY;
                        mx = fmaxf(mx, v);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[i], mx);
                const float base = mn == -INFINITY ? 0.f : mn;
                const float alpha = exp2_fast(m[i] - base);
                m[i] = mn;
                l[i] *= alpha;
#pragma unroll
                for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float& v = s[n][2 * i + c];
                        v = exp2_fast(v - base);
                        l[i] += v;
                    }
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][2 * i] *= alpha;
                    o[n][2 * i + 1] *= alpha;
                }
            }
            // values; P is rounded to the payload type (its error, half a step of a
            // 16-bit type per term, averages out over the terms)
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
                constexpr float w = kWeightUnit<T>;
                unsigned a[4];
                a[0] = f32_to_pair(make_float2(w * s[2 * kk][0], w * s[2 * kk][1]), T());
                a[1] = f32_to_pair(make_float2(w * s[2 * kk][2], w * s[2 * kk][3]), T());
                a[2] = f32_to_pair(make_float2(w * s[2 * kk + 1][0], w * s[2 * kk + 1][1]), T());
                a[3] = f32_to_pair(make_float2(w * s[2 * kk + 1][2], w * s[2 * kk + 1][3]), T());
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    unsigned b[4];
                    ldsm4_t(b, smem_addr(vs + (kk * 16 + (lane & 15)) * P + 32 * n + 16 * (lane >> 4)));
                    mma16816<T>(o[2 * n], a, b[0], b[1]);
                    mma16816<T>(o[2 * n + 1], a, b[2], b[3]);
                }
            }
        }
        copy_wait<0>();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = warp * 16 + (lane >> 2) + 8 * i;
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            // l is 0 only where the row sees nothing (the largest term is 1); NaN stays NaN
            const float inv = l[i] == 0.f ? 0.f : 1.f / (l[i] * kWeightUnit<T>);
            const float lse2 = l[i] == 0.f ? -INFINITY : m[i] + log2f(l[i]);
            if (row >= nrows) continue;
            const int t = q.start + j0 + row / p.gq, h = hkv * p.gq + row % p.gq;
            const int64_t kept = whole ? partial_row(p, q, r, t, h) : (int64_t)slot * kRows + row;
            if (whole && (!kPlanned || kept < 0)) {
                T* out = reinterpret_cast<T*>(p.o + (int64_t)r * p.o_sn + (int64_t)t * p.o_st + (int64_t)h * p.o_sh);
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<unsigned*>(out + n * 8 + (lane & 3) * 2) =
                        f32_to_pair(make_float2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv), T());
                if ((lane & 3) == 0)
                    p.lse[(int64_t)r * p.l_sn + (int64_t)t * p.l_st + (int64_t)h * p.l_sh] =
                        p.base2 ? lse2 : lse2 * kLn2;
            } else {
                float* out = (kPlanned && whole ? partial_o(p) : ws.o) + kept * D;
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(out + n * 8 + (lane & 3) * 2) =
                        make_float2(o[n][2 * i] * inv, o[n][2 * i + 1] * inv);
                if ((lane & 3) == 0) (kPlanned && whole ? partial_lse(p) : ws.lse)[kept] = lse2;
            }
        }
        __syncthreads();
        // what the zeroed values give to the rows that do see them
        unsigned any = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= poison[i >> 1][i & 1];
        if (any && tid < nrows) {
            const int t = q.start + j0 + tid / p.gq, h = hkv * p.gq + tid % p.gq;
            const T* qrow = reinterpret_cast<const T*>(p.q + (int64_t)t * p.q_st + (int64_t)h * p.q_sh);
            const int lm = visible(p, q, j0 + tid / p.gq, r);
            const int64_t at = (int64_t)r * p.l_sn + (int64_t)t * p.l_st + (int64_t)h * p.l_sh;
            const int64_t kept = whole ? partial_row(p, q, r, t, h) : (int64_t)slot * kRows + tid;
            for (int i = 0; i < 4; ++i) {
                if (whole && (!kPlanned || kept < 0))
                    add_nonfinite<T, T>(p, r, table, hkv, qrow, (mtile + i) * kTile, poison[i], 2, lm,
                                        p.base2 ? p.lse[at] : p.lse[at] * kLog2e,
                                        reinterpret_cast<T*>(p.o + (int64_t)r * p.o_sn + (int64_t)t * p.o_st +
                                                             (int64_t)h * p.o_sh));
                else
                    add_nonfinite<T, float>(p, r, table, hkv, qrow, (mtile + i) * kTile, poison[i], 2, lm,
                                            (kPlanned && whole ? partial_lse(p) : ws.lse)[kept],
                                            (kPlanned && whole ? partial_o(p) : ws.o) + kept * D);
            }
        }
        if (cut) break;
        x = next_item(p, x, tpi);
    }
}

int mma_ctas(int D) { return device_sm_count() * (D == 256 ? 2 : 3); }

template <typename T, int D, class Params>
cudaError_t launch_mma(const Params& p, int dtype, cudaStream_t stream) {
    const int ctas = mma_ctas(D), tpi = chunk_attention_mma_tokens(p.gq);
    const ChunkPartials ws = chunk_partials_in(p.ws, ctas, kRows, D);
    constexpr int smem = MmaShape<D>::kSmem;
    const auto kernel = chunk_attention_kernel<T, D, Params>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if constexpr (std::is_same<Params, PrefixParams>::value) {
        e = launch_chained(kernel, ctas, kThreadsMma, smem, stream, p, ws, tpi);
        return e != cudaSuccess ? e : launch_prefix_finish(p, ws, tpi, kRows, ctas, dtype, stream);
    } else {
        kernel<<<ctas, kThreadsMma, smem, stream>>>(p, ws, tpi);
        e = cudaGetLastError();
        return e != cudaSuccess ? e : launch_chunk_merge(p, ws, tpi, kTile, kRows, ctas, dtype, stream);
    }
}

template <typename T, class Params>
cudaError_t launch_mma_d(const Params& p, int dtype, cudaStream_t stream) {
    switch (p.D) {
        case 64: return launch_mma<T, 64>(p, dtype, stream);
        case 128: return launch_mma<T, 128>(p, dtype, stream);
        case 256: return launch_mma<T, 256>(p, dtype, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

size_t chunk_attention_workspace(int N, int B, int T, int H, int Hkv, int D, int max_seq_len) {
    const size_t mma = chunk_partials_bytes(mma_ctas(D), kRows, D), tc = chunk_attention_tc_workspace(D);
    return mma > tc ? mma : tc;
}

cudaError_t launch_chunk_attention(const ChunkParams& p, int dtype, cudaStream_t stream) {
    cudaError_t e;
    if (launch_chunk_attention_tc(p, dtype, stream, &e)) return e;
    return dtype == DCP_F16 ? launch_mma_d<__half>(p, dtype, stream) : launch_mma_d<__nv_bfloat16>(p, dtype, stream);
}

int chunk_attention_mma_tokens(int gq) { return kRows / gq; }

cudaError_t launch_planned_attention(const PrefixParams& p, const void* tc_maps, int dtype, cudaStream_t stream) {
    if (tc_maps) return launch_planned_attention_tc(p, tc_maps, dtype, stream);
    return dtype == DCP_F16 ? launch_mma_d<__half>(p, dtype, stream) : launch_mma_d<__nv_bfloat16>(p, dtype, stream);
}

}  // namespace dcp
