// dcp_chunk_weights.cu -- the attention weights that a ragged batch's new tokens
// give to every cached token, added to the running sums an eviction goes by:
// the register-tiled kernel, which takes every shape.
//
// With the merged log-sum-exp of a row known, a weight is one exponential,
//     w = 2^(s log2e - lse2),  s = sm_scale <q, k>,
// and a token's sum needs no other token: the product runs transposed, S^T =
// K Q^T with the tokens on the rows, so a token's weights lie in one row and
// its sum stays in registers.  The keys are read once; every row of queries
// that sees them passes by.  mma.sync: 64 tokens a CTA, 16 a warp, query rows
// in tiles of 32.  Bound by
// the warp-level products for chunks (183 TFLOP/s: 2048 new tokens over 16384 in
// 1412 us; D = 256 154 TFLOP/s, 3342 us) and by the latency of its loads for single
// tokens (3.8 TB/s; D = 256 3.3 TB/s, 329 us for 64 over 8192).
#include "dcp_chunk.cuh"
#include "dcp_mma.cuh"

namespace dcp {
namespace {

constexpr int kTok = 64;    // tokens of a CTA
constexpr int kQRows = 32;  // query rows of a tile
constexpr int kThreadsW = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsW) chunk_weights_kernel(const ChunkParams p, int tiles) {
    constexpr int P = D * 2 + 16;
    __shared__ __align__(16) unsigned char qs[kQRows * P];
    __shared__ float lse_s[kQRows];
    __shared__ int lim_s[kQRows];
    extern __shared__ __align__(16) unsigned char ks[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x % tiles;
    const int hkv = (blockIdx.x / tiles) % p.Hkv;
    const int rb = blockIdx.x / tiles / p.Hkv;
    const int b = rb % p.B, r = rb / p.B;
    const Request q = load_request(p, b);
    const int held = rank_share(q.L, r, p.N);
    const int tb = tile * kTok;
    if (q.n == 0 || tb >= held) return;
    for (int id = tid; id < kTok * (D / 8); id += kThreadsW) {
        const int row = id / (D / 8), u = id % (D / 8), i = tb + row;
        const int pg = i < held ? page_of(p, r, b, i) : -1;
        copy16(ks + row * P + 16 * u, pg >= 0 ? p.k + k_offset(p, r, pg, i, hkv) + 16 * u : p.k, pg >= 0);
    }
    copy_commit();
    // the first new token that sees the tile: global index tb * N + r or later
    const int jmin = max(0, tb * p.N + r - (q.L - q.n));
    const int m0 = jmin * p.gq, rows = q.n * p.gq;
    const float qscale = p.sm_scale * kLog2e;
    const int my0 = tb + warp * 16 + (lane >> 2);  // this thread's tokens: my0 and my0 + 8
    float sum[2] = {0.f, 0.f};
    for (int mt = m0; mt < rows; mt += kQRows) {
        __syncthreads();
        for (int id = tid; id < kQRows * (D / 8); id += kThreadsW) {
            const int row = mt + id / (D / 8), u = id % (D / 8);
            const bool ok = row < rows;
            const unsigned char* src = p.q;
            if (ok)
                src += (int64_t)(q.start + row / p.gq) * p.q_st + (int64_t)(hkv * p.gq + row % p.gq) * p.q_sh + 16 * u;
            copy16(qs + (row - mt) * P + 16 * u, src, ok);
        }
        copy_commit();
        if (tid < kQRows) {
            const int row = mt + tid;
            float l = 0.f;
            int lim = 0;
            if (row < rows) {
                l = p.lse[(int64_t)(q.start + row / p.gq) * p.l_st + (int64_t)(hkv * p.gq + row % p.gq) * p.l_sh];
                if (!p.base2) l *= kLog2e;
                // a row without a finite log-sum-exp sees nothing
                if (isfinite(l)) lim = visible(p, q, row / p.gq, r);
            }
            lse_s[tid] = l;
            lim_s[tid] = lim;
        }
        copy_wait<0>();
        __syncthreads();
        float s[kQRows / 8][4];
#pragma unroll
        for (int n = 0; n < kQRows / 8; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[n][c] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            unsigned a[4];
            ldsm4(a, smem_addr(ks + (warp * 16 + (lane & 15)) * P + 32 * kk + 16 * (lane >> 4)));
#pragma unroll
            for (int n = 0; n < kQRows / 16; ++n) {
                unsigned bq[4];
                ldsm4(bq,
                      smem_addr(qs + (n * 16 + (lane & 7) + 8 * (lane >> 4)) * P + 32 * kk + 16 * ((lane >> 3) & 1)));
                mma16816<T>(s[2 * n], a, bq[0], bq[1]);
                mma16816<T>(s[2 * n + 1], a, bq[2], bq[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < kQRows / 8; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = n * 8 + (lane & 3) * 2 + c;
                const float l = lse_s[col];
                const int lim = lim_s[col];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float w = exp2_fast(fmaf(s[n][2 * i + c], qscale, -l));
                    if (my0 + 8 * i < lim) sum[i] += w;
                }
            }
    }
    copy_wait<0>();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        const int tok = my0 + 8 * i;
        if ((lane & 3) == 0 && tok < held) {
            float* a = p.acc + (int64_t)r * p.a_sn + (int64_t)b * p.a_sb + (int64_t)hkv * p.a_sh + tok;
            *a = (tok * p.N + r < q.L - q.n ? *a : 0.f) + sum[i];
        }
    }
}

template <typename T, int D>
cudaError_t launch_weights(const ChunkParams& p, cudaStream_t stream) {
    const int64_t cap = ((int64_t)p.max_seq_len + p.N - 1) / p.N;
    const int64_t tiles = (cap + kTok - 1) / kTok;
    if (tiles == 0) return cudaSuccess;
    constexpr int smem = kTok * (D * 2 + 16);
    const cudaError_t e =
        cudaFuncSetAttribute(chunk_weights_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    chunk_weights_kernel<T, D><<<(unsigned)(tiles * p.N * p.B * p.Hkv), kThreadsW, smem, stream>>>(p, (int)tiles);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_weights_d(const ChunkParams& p, cudaStream_t stream) {
    switch (p.D) {
        case 64: return launch_weights<T, 64>(p, stream);
        case 128: return launch_weights<T, 128>(p, stream);
        case 256: return launch_weights<T, 256>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_chunk_weights(const ChunkParams& p, int dtype, cudaStream_t stream) {
    cudaError_t e;
    if (launch_chunk_weights_tc(p, dtype, stream, &e)) return e;
    return dtype == DCP_F16 ? launch_weights_d<__half>(p, stream) : launch_weights_d<__nv_bfloat16>(p, stream);
}

}  // namespace dcp
