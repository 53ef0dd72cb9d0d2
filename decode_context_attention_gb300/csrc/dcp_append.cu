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
// then read once for all of them.  Measured (bf16, 32 query and 4 KV heads of 128):
// 16384 tokens 69 us, 5.0 TB/s (51 us at the copy rate; 4.2 waves of CTAs, DRAM 56% and
// issue slots 62% busy, neither the limit); 64 tokens 4.1 us, of which the launch and
// the look-ups are all.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendCtas = 8;  // per SM: 64 registers a thread, 1024 threads with 64 bytes in flight each

// Eight 16-bit elements as four fp32 pairs (two fp32 operations an instruction:
// with one at a time this kernel was bound by its instructions).
template <typename T>
__device__ __forceinline__ void widen(const uint4& v, Pair (&x)[4]) {
    x[0] = word_to_pair<T>(v.x);
    x[1] = word_to_pair<T>(v.y);
    x[2] = word_to_pair<T>(v.z);
    x[3] = word_to_pair<T>(v.w);
}
template <typename T>
__device__ __forceinline__ uint4 narrow(const Pair (&x)[4]) {
    return make_uint4(f32_to_pair(unpack2(x[0]), T()), f32_to_pair(unpack2(x[1]), T()),
                      f32_to_pair(unpack2(x[2]), T()), f32_to_pair(unpack2(x[3]), T()));
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
    Pair cs[4], sn[4];
    if (turned) {
        const float* c = a.cos_sin + (int64_t)pos * a.rot;
        const int i0 = a.interleaved ? 4 * u : 8 * u;
        const int i1 = a.interleaved ? a.rot / 4 + 4 * u : 8 * u + 4;
        const float4 c0 = __ldg(reinterpret_cast<const float4*>(c + i0));
        const float4 c1 = __ldg(reinterpret_cast<const float4*>(c + i1));
        const float4 s0 = __ldg(reinterpret_cast<const float4*>(c + a.rot / 2 + i0));
        const float4 s1 = __ldg(reinterpret_cast<const float4*>(c + a.rot / 2 + i1));
        cs[0] = pack2f(c0.x, c0.y); cs[1] = pack2f(c0.z, c0.w);
        cs[2] = pack2f(c1.x, c1.y); cs[3] = pack2f(c1.z, c1.w);
        sn[0] = pack2f(s0.x, s0.y); sn[1] = pack2f(s0.z, s0.w);
        sn[2] = pack2f(s1.x, s1.y); sn[3] = pack2f(s1.z, s1.w);
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
            Pair x0[4], x1[4];
            widen<T>(v0, x0);
            widen<T>(v1, x1);
            const unsigned char* w = row < p.H ? a.qw : a.kw;
            if (w) {
                Pair sq = mul2(x0[0], x0[0]), sr = mul2(x1[0], x1[0]);
#pragma unroll
                for (int i = 1; i < 4; ++i) {
                    sq = fma2(x0[i], x0[i], sq);
                    sr = fma2(x1[i], x1[i], sr);
                }
                const float2 f = unpack2(sq), g = unpack2(sr);
                float ss = (f.x + f.y) + (g.x + g.y);
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(gmask, ss, o);
                const float rs = rsqrtf(ss * inv_d + a.eps);
                const Pair rs2 = pack2f(rs, rs);
                Pair w0[4], w1[4];
                widen<T>(mine ? __ldg(reinterpret_cast<const uint4*>(w + 2 * e0)) : zero, w0);
                widen<T>(mine ? __ldg(reinterpret_cast<const uint4*>(w + 2 * e1)) : zero, w1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x0[i] = mul2(mul2(x0[i], rs2), w0[i]);
                    x1[i] = mul2(mul2(x1[i], rs2), w1[i]);
                }
            }
            if (turned) {
                if (a.interleaved) {
                    // pair i of a vector turns by one angle: (a c - b s, b c + a s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 p0 = unpack2(x0[i]), p1 = unpack2(x1[i]);
                        const float2 ca = unpack2(cs[i >> 1]), sa = unpack2(sn[i >> 1]);
                        const float2 cb = unpack2(cs[2 + (i >> 1)]), sb = unpack2(sn[2 + (i >> 1)]);
                        const float c0 = i & 1 ? ca.y : ca.x, s0 = i & 1 ? sa.y : sa.x;
                        const float c1 = i & 1 ? cb.y : cb.x, s1 = i & 1 ? sb.y : sb.x;
                        x0[i] = fma2(x0[i], pack2f(c0, c0), pack2f(-p0.y * s0, p0.x * s0));
                        x1[i] = fma2(x1[i], pack2f(c1, c1), pack2f(-p1.y * s1, p1.x * s1));
                    }
                } else {
                    const Pair minus = pack2f(-1.f, -1.f);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const Pair f = x0[i], g = x1[i];
                        x0[i] = fma2(f, cs[i], mul2(mul2(g, minus), sn[i]));
                        x1[i] = fma2(g, cs[i], mul2(f, sn[i]));
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
