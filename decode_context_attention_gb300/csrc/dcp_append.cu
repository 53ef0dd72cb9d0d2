// dcp_append.cu -- norm of queries and keys per head, rotation by position and
// the append of the new keys and values to the round-robin pages, in one pass.
//
// sglang PR #33926 report, "实现拆解" item 1: rank t % N holds token t.
//
// For a head row x of D elements: y = x w / sqrt(mean x^2 + eps), its first
// rot elements turned in pairs by the position's angle.  Every row is read once
// and written once, so the time is that of the bytes: 2 (H + 2 Hkv) D elements
// of 2 bytes per token.  A group of D / 16 lanes (rounded up to a power of two)
// holds a row, 16 elements a lane as two 16-byte vectors: [8u, 8u + 8) and the
// vector rot / 2 further, so both elements of a rotated pair sit in one lane
// and the sum of squares is the only exchange between lanes.  A group takes
// several rows of one token when there are many tokens: the position's
// cosines and sines, the norm weights and the token's place in the cache are
// then read once for all of them.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendCtas = 8;  // per SM: 64 registers a thread, 1024 threads with 64 bytes in flight each

template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float (&x)[8]) {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(word_to_pair<T>(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&x)[8]) {
    uint4 v;
    v.x = f32_to_pair(make_float2(x[0], x[1]), T());
    v.y = f32_to_pair(make_float2(x[2], x[3]), T());
    v.z = f32_to_pair(make_float2(x[4], x[5]), T());
    v.w = f32_to_pair(make_float2(x[6], x[7]), T());
    return v;
}

// The request that owns row t: the largest b with query_start[b] <= t, -1 when
// t lies before the first or behind the last.  The group's LPR lanes probe as
// many places per step.
template <int LPR>
__device__ __forceinline__ int owner_of(const ChunkParams& p, int t, int u, unsigned gmask, int gshift) {
    int lo = 0, hi = p.B + 1;  // query_start[lo] <= t < query_start[hi], with infinity behind the end
    if (t < __ldg(p.query_start)) return -1;
    while (hi - lo > 1) {
        auto probe = [&](int k) { return lo + 1 + (int)((int64_t)(hi - lo - 1) * (2 * k + 1) / (2 * LPR)); };
        const unsigned le = (__ballot_sync(gmask, __ldg(p.query_start + probe(u)) <= t) & gmask) >> gshift;
        const int n = __popc(le);  // the probes are in order: the first n are <= t
        const int top = n < LPR ? probe(n) : hi;
        if (n) lo = probe(n - 1);
        hi = top;
    }
    return lo < p.B ? lo : -1;
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas) append_kernel(const AppendParams a) {
    const ChunkParams& p = a.c;
    const int lane = threadIdx.x & 31, u = lane % LPR;
    const int gshift = lane - u;
    const unsigned gmask = (LPR == 32 ? 0xffffffffu : ((1u << (LPR % 32)) - 1u)) << gshift;
    const int64_t group = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) / LPR;
    const int gpt = a.groups_per_token;
    const int64_t t64 = group / gpt;
    if (t64 >= p.T) return;  // a whole group leaves together
    const int t = (int)t64;
    const int rows = p.H + 2 * p.Hkv;

    // this lane's two vectors of a row, in elements
    const int nrot = a.rot / 16, nvec = p.D / 16;
    const bool mine = u < nvec, turned = u < nrot;
    const int e0 = turned ? 8 * u : a.rot + 8 * (u - nrot);
    const int e1 = turned ? a.rot / 2 + 8 * u : a.rot + (p.D - a.rot) / 2 + 8 * (u - nrot);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto source = [&](int row) -> const unsigned char* {
        if (row < p.H) return p.q + (int64_t)t * p.q_st + (int64_t)row * p.q_sh;
        if (row < p.H + p.Hkv) return a.kn + (int64_t)t * a.kn_st + (int64_t)(row - p.H) * a.kn_sh;
        return a.vn + (int64_t)t * a.vn_st + (int64_t)(row - p.H - p.Hkv) * a.vn_sh;
    };
    int row = (int)(group % gpt);
    // the first row is on its way while the token's owner is looked up
    uint4 v0 = zero, v1 = zero;
    if (mine && row < rows) {
        const unsigned char* s = source(row);
        v0 = __ldcs(reinterpret_cast<const uint4*>(s + 2 * e0));
        v1 = __ldcs(reinterpret_cast<const uint4*>(s + 2 * e1));
    }
    int pos = 0;
    if (a.rot) pos = __ldg(a.positions + t);
    const int b = owner_of<LPR>(p, t, u, gmask, gshift);
    if (b < 0 || (a.rot && (unsigned)pos >= (unsigned)a.num_positions)) return;
    // place of the token in the caches
    int64_t k_at = -1, v_at = -1;
    {
        const Request q = load_request(p, b);
        const int g = q.L - q.n + (t - q.start);
        if (g >= 0 && g < q.L) {
            const int r = g % p.N, i = g / p.N;
            const int pg = page_of(p, r, b, i);
            if (pg >= 0) {
                k_at = k_offset(p, r, pg, i, 0);
                v_at = v_offset(p, r, pg, i, 0);
            }
        }
    }
    // cosines and sines of this lane's pairs: the same angle for both vectors'
    // elements (halves), or four angles a vector (neighbours)
    float cs[8], sn[8];
    if (turned) {
        const float* c = a.cos_sin + (int64_t)pos * a.rot;
        const int i0 = a.interleaved ? 4 * u : 8 * u;
        const int i1 = a.interleaved ? a.rot / 4 + 4 * u : 8 * u + 4;
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(c + i0));
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(c + i1));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(c + a.rot / 2 + i0));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(c + a.rot / 2 + i1));
        cs[0] = c0.x; cs[1] = c0.y; cs[2] = c0.z; cs[3] = c0.w;
        cs[4] = c1.x; cs[5] = c1.y; cs[6] = c1.z; cs[7] = c1.w;
        sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w;
        sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
    }
    const float inv_d = 1.f / (float)p.D;
    while (row < rows) {
        const int next = row + gpt;
        uint4 n0 = zero, n1 = zero;
        if (mine && next < rows) {  // the next row is in flight while this one is worked on
            const unsigned char* s = source(next);
            n0 = __ldcs(reinterpret_cast<const uint4*>(s + 2 * e0));
            n1 = __ldcs(reinterpret_cast<const uint4*>(s + 2 * e1));
        }
        unsigned char* dst;
        if (row < p.H) {
            dst = a.qo + (int64_t)t * a.qo_st + (int64_t)row * a.qo_sh;
        } else if (row < p.H + p.Hkv) {
            dst = k_at < 0 ? nullptr : p.k + k_at + (int64_t)(row - p.H) * p.k_sh;
        } else {
            dst = v_at < 0 ? nullptr : p.v + v_at + (int64_t)(row - p.H - p.Hkv) * p.v_sh;
        }
        if (row < p.H + p.Hkv) {
            float x0[8], x1[8];
            widen<T>(v0, x0);
            widen<T>(v1, x1);
            const unsigned char* w = row < p.H ? a.qw : a.kw;
            if (w) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(x0[i], x0[i], fmaf(x1[i], x1[i], ss));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
                const float rs = rsqrtf(ss * inv_d + a.eps);
                float w0[8], w1[8];
                widen<T>(mine ? __ldg(reinterpret_cast<const uint4*>(w + 2 * e0)) : zero, w0);
                widen<T>(mine ? __ldg(reinterpret_cast<const uint4*>(w + 2 * e1)) : zero, w1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x0[i] = x0[i] * rs * w0[i];
                    x1[i] = x1[i] * rs * w1[i];
                }
            }
            if (turned) {
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float a0 = x0[2 * i], b0 = x0[2 * i + 1], a1 = x1[2 * i], b1 = x1[2 * i + 1];
                        x0[2 * i] = a0 * cs[i] - b0 * sn[i];
                        x0[2 * i + 1] = b0 * cs[i] + a0 * sn[i];
                        x1[2 * i] = a1 * cs[4 + i] - b1 * sn[4 + i];
                        x1[2 * i + 1] = b1 * cs[4 + i] + a1 * sn[4 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float f = x0[i], s = x1[i];
                        x0[i] = f * cs[i] - s * sn[i];
                        x1[i] = s * cs[i] + f * sn[i];
                    }
                }
            }
            v0 = narrow<T>(x0);
            v1 = narrow<T>(x1);
        }
        if (mine && dst) {
            *reinterpret_cast<uint4*>(dst + 2 * e0) = v0;
            *reinterpret_cast<uint4*>(dst + 2 * e1) = v1;
        }
        row = next;
        v0 = n0;
        v1 = n1;
    }
}

template <typename T, int LPR>
cudaError_t launch_append_t(AppendParams a, cudaStream_t stream) {
    const int rows = a.c.H + 2 * a.c.Hkv;
    // one row a group while that does not yet fill the SMs; then as many rows of a
    // token per group as still do (at least four groups a token).  Measured at
    // 16384 tokens of 32 + 2 x 4 heads of 128: 8 rows 70 us, 4 rows 81 us (the
    // lookups of a token are repeated more often); 64 tokens: 1 row 4.1 us.
    const int64_t full = (int64_t)device_sm_count() * 2048 / LPR;
    int gpt = rows;
    while (gpt > 4 && (int64_t)a.c.T * (gpt / 2) >= full) gpt = (gpt + 1) / 2;
    a.groups_per_token = gpt;
    const int64_t threads = (int64_t)a.c.T * gpt * LPR;
    const int64_t blocks = (threads + kAppendThreads - 1) / kAppendThreads;
    append_kernel<T, LPR><<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append_d(const AppendParams& a, cudaStream_t stream) {
    const int v = a.c.D / 16;
    if (v <= 1) return launch_append_t<T, 1>(a, stream);
    if (v <= 2) return launch_append_t<T, 2>(a, stream);
    if (v <= 4) return launch_append_t<T, 4>(a, stream);
    if (v <= 8) return launch_append_t<T, 8>(a, stream);
    if (v <= 16) return launch_append_t<T, 16>(a, stream);
    return launch_append_t<T, 32>(a, stream);
}

}  // namespace

cudaError_t launch_append(const AppendParams& a, int dtype, cudaStream_t stream) {
    return dtype == DCP_F16 ? launch_append_d<__half>(a, stream) : launch_append_d<__nv_bfloat16>(a, stream);
}

}  // namespace dcp
