// dcp_prefix.cu -- the attention of a batch whose requests share long prefixes: the
// plan in front of the chunk-attention kernels, and the join behind them.
//
// sglang PR #34213 report, "功能与动机": partial results over disjoint tokens are
// joined by their log-sum-exps; what that merge does over ranks is done here over the
// tokens that a group of requests has in common and those of each request:
//     lse = log(e^lse_c + e^lse_o),  o = e^(lse_c - lse) o_c + e^(lse_o - lse) o_o.
//
// The plan turns B requests in G groups into G + B requests of the chunk attention: the
// rows of a whole group over the common pages, not causal, and every request's rows
// over its own pages.  A common part is a multiple of N * page_size tokens, so what is
// left of a request is again a request over round-robin pages, from a later entry of
// its table on.  Common keys and values are so read once for up to 256 rows, instead of
// once a request; both kinds of parts go through one launch, cut into equal ranges.
// Parts that are joined leave fp32 rows (8 bytes an element and side more than the
// output alone; a request without a common part writes its output directly).
#include "dcp_chunk.cuh"
#include "dcp_groups.cuh"

namespace dcp {
namespace {

constexpr int kPlanThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void put(const PrefixParams& p, int v, int start, int n, int L, int b, int first, int kind,
                                    int common) {
    p.plan[2 * (int64_t)v] = make_int4(start, n, L, b);
    p.plan[2 * (int64_t)v + 1] = make_int4(first, kind, common, 0);
}

// One CTA a group, then CTAs for the requests outside of groups.  Every entry of the
// plan is written whatever the groups' arrays hold: a request belongs to the group that
// group_of finds, or to none.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixParams p) {
    const ChunkParams& c = p;
    const Groups groups = {p.groups, p.group_start, p.prefix_lens, p.N, p.page_shift, p.max_seq_len, p.max_pages};
    const int tid = threadIdx.x;
    if ((int)blockIdx.x >= p.groups) {
        const int step = (gridDim.x - p.groups) * kPlanThreads;
        for (int b = (blockIdx.x - p.groups) * kPlanThreads + tid; b < p.requests; b += step) {
            if (group_of(groups, b) >= 0) continue;
            const Request q = load_request(c, b);
            put(p, p.groups + b, q.start, q.n, q.L, b, 0, kAlone, 0);
        }
        return;
    }
    __shared__ int least, active, entries;
    const int g = blockIdx.x;
    const int b0 = min(max(__ldg(p.group_start + g), 0), p.requests);
    const int b1 = min(max(__ldg(p.group_start + g + 1), b0), p.requests);
    if (tid == 0) {
        least = p.max_seq_len;
        active = 0;
    }
    __syncthreads();
    // tokens that every new token of the group sees
    int low = p.max_seq_len, count = 0;
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        const Request q = load_request(c, b);
        if (q.n == 0 || group_of(groups, b) != g) continue;
        low = min(low, p.causal ? q.L - q.n : q.L);
        ++count;
    }
    low = __reduce_min_sync(kAll, low);
    count = __reduce_add_sync(kAll, count);
    if ((tid & 31) == 0) {
        atomicMin(&least, low);
        atomicAdd(&active, count);
    }
    __syncthreads();
    if (tid == 0) {
        int common = min(common_entries(groups, g), (max(least, 0) / p.N) >> p.page_shift);
        if (active < 2) common = 0;
        entries = common;
        const Request x = load_request(c, min(b0, p.requests - 1)), y = load_request(c, max(b1 - 1, 0));
        put(p, g, x.start, common ? max(y.start + y.n - x.start, 0) : 0, (common << p.page_shift) * p.N, b0, 0, kCommon, 0);
    }
    __syncthreads();
    const int common = entries, tokens = (common << p.page_shift) * p.N;
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        if (group_of(groups, b) != g) continue;
        const Request q = load_request(c, b);
        // (a request without new tokens may hold less than the common part, and asks for nothing)
        put(p, p.groups + b, q.start, q.n, max(q.L - tokens, 0), b, common, common ? kOwn : kAlone, g);
    }
}

// Rows of a part: their fp32 outputs and base-2 log-sum-exps, one after the other.
struct Rows {
    const float* o;
    const float* l;
};

constexpr int kJoinRows = 4;   // heads of a warp
constexpr int kJoinWarps = 8;
constexpr int kMaxRanges = 1024;

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_kernel(const PrefixParams p, const ChunkPartials ws,
                                                                      int tpi, int rows, int ctas) {
    constexpr int NV = (D + 127) / 128;  // 16-byte vectors of a lane
    __shared__ ChunkPos pos[kMaxRanges + 1];
    for (int c = threadIdx.x; c <= ctas; c += 32 * kJoinWarps) pos[c] = ws.pos[c];
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const int quads = (p.gq + kJoinRows - 1) / kJoinRows;
    const int tokens = min(max(__ldg(p.query_start + p.requests), 0), p.T);
    const int64_t tasks = (int64_t)tokens * p.N * p.Hkv * quads;
    for (int64_t task = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5); task < tasks;
         task += (int64_t)gridDim.x * kJoinWarps) {
        const int h0 = (int)(task % quads) * kJoinRows;
        const int64_t rest = task / quads;
        const int rh = (int)(rest % (p.N * p.Hkv)), t = (int)(rest / (p.N * p.Hkv));
        const int r = rh / p.Hkv, hkv = rh - r * p.Hkv;
        const int nrows = min(kJoinRows, p.gq - h0);
        // the request of token t: the last one that starts at or before it
        int lo = 0, hi = p.requests;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
            const int n = __popc(__ballot_sync(kAll, at < hi && __ldg(p.query_start + at) <= t));
            hi = min(hi, lo + (n + 1) * step);
            lo += n * step;
        }
        const Planned own = load_request(p, p.groups + lo);
        if (t < own.start || t >= own.start + own.n) continue;  // of no request
        // the range that holds the first tile of the item, and whether the next one begins inside it
        int c = 0;
        bool cut = false;
        ChunkPos item;
        auto find = [&](int v, const Planned& q) {
            item = {v, rh, (t - q.start) / tpi, 0};
            int n = 0;
            for (int k = lane; k <= ctas; k += 32) {
                const ChunkPos x = pos[k];
                const bool before = x.b != item.b ? x.b < item.b
                                    : x.rh != item.rh ? x.rh < item.rh
                                    : x.qt != item.qt ? x.qt < item.qt : x.tile == 0;
                n += before ? 1 : 0;
            }
            c = __reduce_add_sync(kAll, n) - 1;
            cut = c < ctas && same_item(pos[c + 1], item);
        };
        const bool joined = own.kind == kOwn;
        Planned q = joined ? load_request(p, own.common) : own;
        if (t < q.start || t >= q.start + q.n) continue;
        bool last = !joined;
        find(joined ? own.common : p.groups + lo, q);
        if (last && !cut) continue;  // written by the kernel itself
        int row = 0;
        int64_t whole = 0;
        auto where = [&]() {  // the item's rows of these heads, and the plan's
            row = (t - q.start - item.qt * tpi) * p.gq + h0;
            whole = partial_row(p, q, r, t, hkv * p.gq + h0);
        };
        where();
        bool begin = true, done = false;
        auto next = [&]() -> Rows {
            for (;;) {
                if (done) return {nullptr, nullptr};
                if (begin) {
                    begin = false;
                    if (!cut) {
                        const Rows x = {p.wo + whole * D, p.wl + whole};
                        c = ctas;  // nothing behind it
                        return x;
                    }
                    const int64_t at = (int64_t)(2 * c + (same_item(pos[c], item) ? 0 : 1)) * rows + row;
                    ++c;
                    return {ws.o + at * D, ws.lse + at};
                }
                if (c < ctas && same_item(pos[c], item)) {
                    const bool empty = same_item(pos[c + 1], item) && pos[c + 1].tile == pos[c].tile;
                    const int64_t at = (int64_t)(2 * c) * rows + row;
                    ++c;
                    if (!empty) return {ws.o + at * D, ws.lse + at};
                    continue;
                }
                if (last) {
                    done = true;
                } else {
                    last = true;
                    begin = true;
                    q = own;
                    find(p.groups + lo, q);
                    where();
                }
            }
        };
        float mx[kJoinRows], sum[kJoinRows];
        float4 acc[kJoinRows][NV];
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            mx[k] = -INFINITY;
            sum[k] = 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) acc[k][v] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // two parts at a time, all their rows in flight
        for (Rows x[2] = {next(), next()}; x[0].o; x[0] = next(), x[1] = next()) {
            float w[2][kJoinRows];
            float4 o[2][kJoinRows][NV];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < kJoinRows; ++k) {
                    const bool ok = x[e].o && k < nrows;
                    w[e][k] = ok ? x[e].l[k] : -INFINITY;
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        o[e][k][v] = ok && 4 * lane + 128 * v < D
                                         ? *reinterpret_cast<const float4*>(x[e].o + k * D + 4 * lane + 128 * v)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int k = 0; k < kJoinRows; ++k) {
                // mx becomes finite, infinite or NaN with the parts: as the formula has it
                const float m = fmaxf(mx[k], fmaxf(w[0][k], w[1][k]));
                const float old = mx[k] == -INFINITY ? 0.f : exp2f(mx[k] - m);
                const float w0 = w[0][k] == -INFINITY ? 0.f : exp2f(w[0][k] - m);
                const float w1 = w[1][k] == -INFINITY ? 0.f : exp2f(w[1][k] - m);
                mx[k] = m;
                sum[k] = fmaf(sum[k], old, w0 + w1);
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    float4& a = acc[k][v];
                    const float4 &o0 = o[0][k][v], &o1 = o[1][k][v];
                    a.x = fmaf(w1, o1.x, fmaf(w0, o0.x, a.x * old));
                    a.y = fmaf(w1, o1.y, fmaf(w0, o0.y, a.y * old));
                    a.z = fmaf(w1, o1.z, fmaf(w0, o0.z, a.z * old));
                    a.w = fmaf(w1, o1.w, fmaf(w0, o0.w, a.w * old));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kJoinRows; ++k) {
            if (k >= nrows) break;
            const float inv = sum[k] == 0.f ? 0.f : 1.f / sum[k];
            const int h = hkv * p.gq + h0 + k;
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
}

template <typename T>
cudaError_t launch_join(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas,
                        cudaStream_t stream) {
    const auto kernel = p.D == 64 ? prefix_join_kernel<T, 64>
                                  : p.D == 128 ? prefix_join_kernel<T, 128> : prefix_join_kernel<T, 256>;
    const int64_t tasks = (int64_t)p.T * p.N * p.Hkv * ((p.gq + kJoinRows - 1) / kJoinRows);
    const int64_t blocks = (tasks + kJoinWarps - 1) / kJoinWarps, most = 4ll * device_sm_count();
    kernel<<<(unsigned)(blocks < most ? blocks : most), 32 * kJoinWarps, 0, stream>>>(p, ws, tpi, rows, ctas);
    return cudaGetLastError();
}

constexpr size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

cudaError_t launch_prefix_join(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                               cudaStream_t stream) {
    if (ctas > kMaxRanges) return cudaErrorInvalidValue;
    return dtype == DCP_F16 ? launch_join<__half>(p, ws, tpi, rows, ctas, stream)
                            : launch_join<__nv_bfloat16>(p, ws, tpi, rows, ctas, stream);
}

// The chunk kernels' partials, the plan, and the rows that are joined.
size_t prefix_attention_workspace(int N, int B, int T, int H, int Hkv, int D, int max_seq_len, int G) {
    const size_t parts = align256(chunk_attention_workspace(N, B, T, H, Hkv, D, max_seq_len));
    if (!G) return parts;
    const size_t rows = (size_t)2 * N * T * H;
    return parts + align256((size_t)32 * ((size_t)G + B)) + align256(rows * D * 4) + align256(rows * 4);
}

cudaError_t launch_prefix_attention(PrefixParams p, int dtype, cudaStream_t stream) {
    if (!p.groups) return launch_chunk_attention(p, dtype, stream);
    unsigned char* at = p.ws + align256(chunk_attention_workspace(p.N, p.requests, p.T, p.H, p.Hkv, p.D, p.max_seq_len));
    p.plan = reinterpret_cast<int4*>(at);
    at += align256((size_t)32 * ((size_t)p.groups + p.requests));
    const size_t rows = (size_t)2 * p.N * p.T * p.H;
    p.wo = reinterpret_cast<float*>(at);
    p.wl = reinterpret_cast<float*>(at + align256(rows * p.D * 4));
    p.B = p.groups + p.requests;
    const int rest = (p.requests + kPlanThreads - 1) / kPlanThreads, most = device_sm_count();
    prefix_plan_kernel<<<p.groups + (rest < most ? rest : most), kPlanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_planned_attention(p, dtype, stream);
}

}  // namespace dcp
