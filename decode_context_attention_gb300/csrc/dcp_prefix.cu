// dcp_prefix.cu -- the attention of a batch whose requests share long prefixes: the
// plan in front of the chunk-attention kernels.
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
// its table on.  Common keys and values are so read once for up to 256 rows (64 in the
// register-tiled kernel), instead of once a request; both kinds of parts go through one
// launch, cut into equal ranges.  Parts that are joined leave fp32 rows; a request that
// shares nothing is written as the chunk attention writes it.
// A request's own part of few rows and tokens (a decode step's) is no work for the
// tensor-core kernel, whose items cost 5 us of an SM each whatever their size: it is
// left to the kernel of dcp_prefix_finish.cu, which joins it with its common part.
// (64 single tokens behind 32768 on 4 ranks: 164 us without that kernel, 88 with it; 256
// behind 2048: 313 and 80.)
// Plan, parts and join are three kernels, each started while the one before ends.
#include <cuda.h>

#include "dcp_chunk.cuh"
#include "dcp_groups.cuh"

namespace dcp {
namespace {

constexpr int kPlanThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ void put(int4* at, int start, int n, int L, int b, int first, int kind, int common) {
    at[0] = make_int4(start, n, L, b);
    at[1] = make_int4(first, kind, common, 0);
}
// Request b's own part, L tokens from entry `first` on, to the one kernel or the other.
__device__ __forceinline__ void put_own(const PrefixParams& p, const Request& q, int L, int b, int first, int kind,
                                        int common, int slim_tokens) {
    const bool slim = q.n * p.gq <= p.slim_rows && rank_share(L, 0, p.N) <= slim_tokens;
    put(p.plan + 2 * (int64_t)b, q.start, slim ? 0 : q.n, L, b, first, kind, p.requests + common);
    put(p.slim + 2 * (int64_t)b, q.start, slim ? q.n : 0, L, b, first, kind, p.requests + common);
}

// Whether the whole batch is so little work that the kernel of the slim parts does all of it
// sooner, prefixes read once a request, than the chunk kernel starts and ends: requests of
// few rows, up to kSmallTokens of a rank each, and kSmallTiles tiles of 128 tokens and up to
// 128 columns in all (a tile is 1.2 us of an SM; chosen on 152 SMs, and not scaled with
// their number).  All CTAs come to the same answer.
// Replayed: 23 requests behind up to 1850 tokens on 3 ranks 33 us with the chunk kernel, 25
// without; 18 behind 157 19 and 15; but 91 behind 998, of 2900 tiles, 36 and 42, and with
// 2048 tokens of a rank one request's tiles outlast the chunk kernel (8 behind 1300 27 and 37).
constexpr int kSmallRequests = 4096;
constexpr int kSmallTokens = 1024;
constexpr int64_t kSmallTiles = 1900;
__device__ __forceinline__ bool small_batch(const PrefixParams& p, int* scratch) {
    if (p.slim_rows == 0 || p.requests > kSmallRequests) return false;
    const ChunkParams& c = p;
    if (threadIdx.x == 0) *scratch = 0;
    __syncthreads();
    int tiles = 0, wide = 0;
    for (int b = threadIdx.x; b < p.requests; b += kPlanThreads) {
        const Request q = load_request(c, b);
        const int tokens = rank_share(q.L, 0, p.N);
        if (q.n == 0) continue;
        wide |= q.n * p.gq > p.slim_rows || tokens > kSmallTokens;
        tiles += tokens / 128 + 1;  // at most 9 a request
    }
    tiles = (int)__reduce_add_sync(kAll, (unsigned)tiles);
    if ((threadIdx.x & 31) == 0) atomicAdd(scratch, tiles);
    wide = __syncthreads_or(wide);
    return !wide && (int64_t)*scratch * p.N * p.Hkv * (p.D == 256 ? 2 : 1) <= kSmallTiles;
}

// One CTA a group, then CTAs for the requests outside of groups.  Every entry of the
// plan is written whatever the groups' arrays hold: a request belongs to the group that
// group_of finds, or to none.
__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixParams p) {
    const ChunkParams& c = p;
    const Groups groups = {p.groups, p.group_start, p.prefix_lens, p.N, p.page_shift, p.max_seq_len, p.max_pages};
    const int tid = threadIdx.x;
    __shared__ int scratch;
    chain_release();
    const bool small = small_batch(p, &scratch);
    const int slim_tokens = small ? kSmallTokens : p.slim_tokens;
    if (blockIdx.x == 0 && tid == 0) *p.nothing = small;
    if ((int)blockIdx.x >= p.groups) {
        const int step = (gridDim.x - p.groups) * kPlanThreads;
        for (int b = (blockIdx.x - p.groups) * kPlanThreads + tid; b < p.requests; b += step) {
            if (group_of(groups, b) >= 0) continue;
            const Request q = load_request(c, b);
            put_own(p, q, q.L, b, 0, kAlone, 0, slim_tokens);
        }
        return;
    }
    __shared__ int least, tokens_new, blocks, slim, entries, asks;
    const int g = blockIdx.x;
    const int b0 = min(max(__ldg(p.group_start + g), 0), p.requests);
    const int b1 = min(max(__ldg(p.group_start + g + 1), b0), p.requests);
    if (tid == 0) {
        least = p.max_seq_len;
        tokens_new = blocks = slim = 0;
        asks = p.requests;
    }
    __syncthreads();
    // tokens that every new token of the group sees, the first request that brings one, the blocks of rows that
    // the requests are alone, and the requests of few rows
    int low = p.max_seq_len, at = p.requests, sums[3] = {0, 0, 0};
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        const Request q = load_request(c, b);
        if (q.n == 0 || group_of(groups, b) != g) continue;
        low = min(low, p.causal ? q.L - q.n : q.L);
        at = min(at, b);
        sums[0] += q.n;
        if (q.n * p.gq <= p.slim_rows) ++sums[2];
        else sums[1] += (q.n + p.plan_tpi - 1) / p.plan_tpi;
    }
    low = __reduce_min_sync(kAll, low);
    at = __reduce_min_sync(kAll, at);
#pragma unroll
    for (int e = 0; e < 3; ++e) sums[e] = (int)__reduce_add_sync(kAll, (unsigned)sums[e]);
    if ((tid & 31) == 0) {
        atomicMin(&least, low);
        atomicMin(&asks, at);
        atomicAdd(&tokens_new, sums[0]);
        atomicAdd(&blocks, sums[1]);
        atomicAdd(&slim, sums[2]);
    }
    __syncthreads();
    if (tid == 0) {
        int common = min(common_entries(groups, g), (max(least, 0) / p.N) >> p.page_shift);
        // In the chunk kernel's units of work (0.4 us of an SM; a tile of 128 tokens is 4, an item 13): what a
        // request's tiles cost it alone, less what its own part costs as an item more and a row to be joined
        // (30; a slim part's tiles 3, as a kernel of their own reads them), against the common part's.
        // 8 chunks of 512 tokens of 8 heads a group, which fill blocks of rows by themselves: 1153 us shared,
        // 796 alone; 64 single tokens: 118 shared, 541 alone.
        const int64_t tiles8 = ((int64_t)common << p.page_shift) / 16;  // in eighths
        const int64_t shared = (tokens_new + p.plan_tpi - 1) / p.plan_tpi;
        if (blocks * (4 * tiles8 - 8 * 30) + 3 * tiles8 * slim <= shared * (8 * 13 + 4 * tiles8) || small)
            common = 0;
        entries = common;
        const Request x = load_request(c, min(b0, p.requests - 1)), y = load_request(c, max(b1 - 1, 0));
        // by the entries of the group's first request if it holds that many tokens, else of the first that asks,
        // which does: a request without new tokens may hold less, and its entries then name nothing
        const int tokens = (common << p.page_shift) * p.N;
        put(p.plan + 2 * ((int64_t)p.requests + g), x.start, common ? max(y.start + y.n - x.start, 0) : 0, tokens,
            x.L < tokens ? min(asks, p.requests - 1) : b0, 0, kCommon, 0);
    }
    __syncthreads();
    const int common = entries, tokens = (common << p.page_shift) * p.N;
    for (int b = b0 + tid; b < b1; b += kPlanThreads) {
        if (group_of(groups, b) != g) continue;
        const Request q = load_request(c, b);
        // (a request without new tokens may hold less than the common part, and asks for nothing)
        put_own(p, q, max(q.L - tokens, 0), b, common, common ? kOwn : kAlone, g,
                slim_tokens);
    }
}

constexpr size_t align256(size_t n) { return (n + 255) & ~size_t(255); }
// CTAs for the requests outside of groups.
int plan_rest(int B) {
    const int rest = (B + kPlanThreads - 1) / kPlanThreads;
    return rest < 128 ? rest : 128;
}

}  // namespace

// The chunk kernels' partials, the plan, and the rows that are joined.
size_t prefix_attention_workspace(int N, int B, int T, int H, int Hkv, int D, int max_seq_len, int G) {
    const size_t chunk = chunk_attention_workspace(N, B, T, H, Hkv, D, max_seq_len);
    if (!G) return chunk;
    const size_t parts = align256(chunk) + 256;  // (from the workspace's first 256-byte boundary on)
    const size_t rows = (size_t)2 * N * T * H;
    return parts + align256((size_t)32 * ((size_t)G + 2 * (size_t)B) + 32) +
           align256(rows * D * 4) + align256(rows * 4);
}

cudaError_t launch_prefix_attention(PrefixParams p, int dtype, cudaStream_t stream) {
    if (!p.groups) return launch_chunk_attention(p, dtype, stream);
    p.ws = reinterpret_cast<unsigned char*>(align256((size_t)p.ws));
    unsigned char* at = p.ws + align256(chunk_attention_workspace(p.N, p.requests, p.T, p.H, p.Hkv, p.D, p.max_seq_len));
    p.plan = reinterpret_cast<int4*>(at);
    p.slim = p.plan + 2 * ((size_t)p.groups + p.requests);
    p.nothing = reinterpret_cast<int*>(p.slim + 2 * (size_t)p.requests);
    at += align256((size_t)32 * ((size_t)p.groups + 2 * (size_t)p.requests) + 32);
    const size_t rows = (size_t)2 * p.N * p.T * p.H;
    p.wo = reinterpret_cast<float*>(at);
    p.wl = reinterpret_cast<float*>(at + align256(rows * p.D * 4));
    p.B = p.groups + p.requests;
    CUtensorMap maps[2], tc_maps[3];
    slim_limits(p, dtype, maps);
    // the sharing rule counts blocks of rows as the kernel cuts them that will run
    const bool tc = planned_attention_tc_maps(p, dtype, tc_maps);
    p.plan_tpi = tc ? chunk_attention_tc_tokens(p.gq) : chunk_attention_mma_tokens(p.gq);
    prefix_plan_kernel<<<p.groups + plan_rest(p.requests), kPlanThreads, 0, stream>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_planned_attention(p, tc ? tc_maps : nullptr, dtype, stream);
}

}  // namespace dcp
