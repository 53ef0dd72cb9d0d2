// dcp_pages.cu -- the bookkeeping of round-robin paged caches on the device: a
// step's index arrays and the pages of its new tokens from the requests' lengths,
// and the way of pages back to the ranks' free lists.
//
// sglang PR #33926 report, "关键源码片段" (`get_dcp_lens`): rank r holds n / N of
// n tokens, one more when r < n % N; "实现拆解" item 1 builds the tables over that
// slice.  The pages build them on the host; here lengths never leave the device, so
// a captured step stays valid while requests grow.
//
// With share(n, r) = n / N + (r < n % N) and S the entries a request has in common
// with its group's first one, request b needs new pages for the entries
//     [max(ceil(share(cached, r) / page), S), ceil(share(cached + n, r) / page))
// of rank r's row.  The k-th entry of a rank, counted over the requests in order, takes
// the k-th page from the top of the rank's stack.  Entry numbers are sums over the
// requests before: one scan of the new tokens, then one of the entries, by the CTAs of a
// cluster for a rank.  Everything else (common entries, the tokens' arrays) follows from
// the scans' results entry by entry.
//
// All of it is latency: a launch, and a chain of loads, scans and barriers.  Replayed,
// 64 requests of one token take 8.2 us, 16384 tokens of 8 requests 10.3, 4096 requests on
// 8 ranks 16.5 (one CTA a rank: 27); pages of 64 requests given back 8.2, of a fifth of
// 4096 10.5 (one CTA a rank: 25).  A call from Python takes 12 to 24, its arguments' checks.
#include "dcp_chain.cuh"
#include "dcp_groups.cuh"
#include "dcp_internal.h"
#include "dcp_sm100.cuh"

namespace dcp {
namespace {

constexpr int kThreadsPages = 1024;

__device__ __forceinline__ int share_of(int n, int r, int N) { return n / N + (r < n % N ? 1 : 0); }
// Table entries that n tokens take on rank r.
__device__ __forceinline__ int entries_of(const PageParams& p, int n, int r) {
    return (int)(((int64_t)share_of(n, r, p.N) + (1 << p.page_shift) - 1) >> p.page_shift);
}
__device__ __forceinline__ Groups groups_of(const PageParams& p) {
    return {p.G, p.group_start, p.prefix_lens, p.N, p.page_shift, p.max_seq_len, p.max_pages};
}
__device__ __forceinline__ int cached_of(const PageParams& p, int b) {
    return min(max(__ldg(p.cached_lens + b), 0), p.max_seq_len);
}
// Pages on rank r's stack.  (A plain load: free_out may be free_count, and a read-only one may be made again after
// the count has been written.)
__device__ __forceinline__ int pages_free(const PageParams& p, int r) {
    return min(max(p.free_count[r], 0), p.free_capacity);
}

// Inclusive sum over the block's threads; `warps` holds 32 numbers, free again
// after the next barrier.  Ends behind a barrier.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warps, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) warps[warp] = v;
    __syncthreads();
    int64_t w = lane < (int)(blockDim.x >> 5) ? warps[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    if (warp) v += __shfl_sync(0xffffffffu, w, warp - 1);
    __syncthreads();
    return v;
}

// The sum of `v` over the CTAs of this one's cluster before it, and over all `ctas`.  All
// threads; `turn` counts the calls, whose barriers keep a value until everyone has it.
struct Exchange {
    int64_t of[2];
};
__device__ __forceinline__ int64_t sum_before(int64_t v, Exchange* x, int ctas, int turn, int64_t* total) {
    *total = v;
    if (ctas == 1) return 0;
    if (threadIdx.x == 0) x->of[turn & 1] = v;
    sm100::cluster_sync();
    const int me = (int)sm100::cluster_ctarank();
    int64_t before = 0, all = 0;
    for (int k = 0; k < ctas; ++k) {
        int64_t y;
        asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.b64 %0, [a];\n}"
                     : "=l"(y)
                     : "r"(sm100::smem_u32(&x->of[turn & 1])), "r"(k));
        all += y;
        if (k < me) before += y;
    }
    *total = all;
    return before;
}

// The last index i of [0, n) with at[i] <= x, for at[0] <= x and `at` non-decreasing.
template <typename I>
__device__ __forceinline__ int last_at_or_before(const I* at, int n, I x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Lengths, and rank r's new pages, by CTA `cta` of `ctas`: a cluster's, or one alone.
__device__ void reserve_rank(const PageParams& p, const Groups& groups, int r, bool lengths, int cta, int ctas) {
    __shared__ int64_t warps[32];
    __shared__ int64_t off[kThreadsPages];
    __shared__ int have[kThreadsPages];
    __shared__ Exchange exchange;
    const int tid = threadIdx.x;
    const int left = pages_free(p, r);
    const int* free = p.free_pages + (int64_t)r * p.fp_sn;
    int* row = p.bt + (int64_t)r * p.bt_sn;
    int64_t rows = 0, used = 0;  // new tokens and entries of the requests before
    int turn = 0;
    if (lengths && cta == 0 && tid == 0) p.query_start[0] = 0;
    // requests of a CTA at a time, so that all have some
    const int per = min((p.B + ctas - 1) / ctas, kThreadsPages);
    for (int64_t first = 0; first < p.B; first += (int64_t)per * ctas) {
        const int64_t b0 = first + (int64_t)cta * per, b = b0 + tid;
        const bool there = tid < per && b < p.B;
        const int cached = there ? cached_of(p, (int)b) : 0;
        int n = there ? min(max(__ldg(p.new_lens + b), 0), p.max_seq_len - cached) : 0;
        int64_t total;
        // token rows end at T: what does not fit is cut off
        int64_t end = rows + block_scan(n, warps, &total);
        end += sum_before(total, &exchange, ctas, turn++, &total);
        const int s1 = (int)min(end, (int64_t)p.T), s0 = (int)min(end - n, (int64_t)p.T);
        n = s1 - s0;
        rows = min(rows + total, (int64_t)p.T);
        if (there && lengths) {
            p.query_start[b + 1] = s1;
            p.seq_lens[b] = cached + n;
        }
        int low = 0, count = 0;
        if (there) {
            low = max(entries_of(p, cached, r), p.G ? member_of(groups, (int)b).entries : 0);
            count = max(entries_of(p, cached + n, r) - low, 0);
        }
        const int64_t upto = block_scan(count, warps, &total);
        off[tid] = upto - count;
        have[tid] = low;
        const int64_t mine = total;
        const int64_t before = used + sum_before(total, &exchange, ctas, turn++, &total);
        __syncthreads();
        for (int64_t k = tid; k < mine; k += kThreadsPages) {
            const int i = last_at_or_before(off, kThreadsPages, k);
            const int64_t at = left - 1 - (before + k);
            row[(b0 + i) * p.bt_sb + have[i] + (k - off[i])] = at >= 0 ? __ldg(free + at) : -1;
        }
        used += total;
        __syncthreads();
    }
    if (cta == 0 && tid == 0) {
        p.free_out[r] = (int)max(left - used, (int64_t)0);
        p.missing[r] = (int)min(max(used - left, (int64_t)0), (int64_t)0x7fffffff);
    }
    if (ctas > 1) sm100::cluster_sync();  // a CTA's sums are read until here
}

// Common entries and the tokens' arrays, by worker `worker` of `workers` threads (whole
// warps), from what reserve_rank left in memory.
__device__ __forceinline__ void reserve_rest(const PageParams& p, const Groups& groups, int64_t worker,
                                             int64_t workers) {
    const int lane = (int)(worker & 31);
    if (p.G) {
        // eight lanes a (request, rank): its common entries are some tens
        for (int64_t pair = worker >> 3; pair < (int64_t)p.N * p.B; pair += workers >> 3) {
            const int b = (int)(pair / p.N), r = (int)(pair - (int64_t)b * p.N);
            const Member m = member_of(groups, b);
            const int* from = p.bt + (int64_t)r * p.bt_sn + (int64_t)m.first * p.bt_sb;
            int* to = p.bt + (int64_t)r * p.bt_sn + (int64_t)b * p.bt_sb;
            for (int j = lane & 7; j < m.entries; j += 8) to[j] = from[j];
        }
    }
    if (!p.positions && !p.slots && !p.requests) return;
    const int n = p.query_start[p.B];
    for (int64_t t0 = worker - lane; t0 < n; t0 += workers) {
        // the requests of the warp's first and last token, by 32 places at a time; between them each lane's own
        auto request_of = [&](int token, int lo) {
            int hi = p.B;  // query_start[lo] <= token; requests from hi on start behind it
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
                const int before = __popc(__ballot_sync(0xffffffffu, at < hi && p.query_start[min(at, p.B)] <= token));
                hi = min(hi, lo + (before + 1) * step);
                lo += before * step;
            }
            return lo;
        };
        const int first = request_of((int)t0, 0), last = request_of(min((int)t0 + 31, n - 1), first);
        const int t = (int)t0 + lane;
        if (t >= n) continue;
        const int b = first + last_at_or_before(p.query_start + first, last - first + 1, t);
        const int g = cached_of(p, b) + t - p.query_start[b];
        if (p.positions) p.positions[t] = g;
        if (p.requests) p.requests[t] = b;
        if (p.slots) {
            const int r = g % p.N, i = g / p.N, j = i >> p.page_shift;
            // a common entry is read where it comes from, whether or not its copy is made yet
            int from = b;
            if (p.G) {
                const Member m = member_of(groups, b);
                if (j < m.entries) from = m.first;
            }
            const int pg = p.bt[(int64_t)r * p.bt_sn + (int64_t)from * p.bt_sb + j];
            p.slots[t] = (unsigned)pg < (unsigned)p.num_pages
                             ? ((((int64_t)r * p.num_pages + pg) << p.page_shift) | (i & ((1 << p.page_shift) - 1)))
                             : -1;
        }
    }
}

// All of a small call by one cluster, whose barrier stands between the two steps.
constexpr int kCluster = 8;
__global__ void __launch_bounds__(kThreadsPages) reserve_small_kernel(const PageParams p) {
    __shared__ GroupsHeld held;
    const Groups groups = hold_groups(groups_of(p), &held);
    const int cta = blockIdx.x;
    for (int r = cta; r < p.N; r += kCluster) reserve_rank(p, groups, r, r == 0, 0, 1);
    sm100::cluster_sync();
    reserve_rest(p, groups, cta * kThreadsPages + threadIdx.x, kCluster * kThreadsPages);
}
__global__ void __launch_bounds__(kThreadsPages) reserve_pages_kernel(const PageParams p, int ctas) {
    __shared__ GroupsHeld held;
    chain_release();
    const int r = blockIdx.x / ctas;
    reserve_rank(p, hold_groups(groups_of(p), &held), r, r == 0, blockIdx.x - r * ctas, ctas);
}
__global__ void __launch_bounds__(256) reserve_rest_kernel(const PageParams p) {
    __shared__ GroupsHeld held;
    const Groups groups = hold_groups(groups_of(p), &held);
    chain_wait();
    reserve_rest(p, groups, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// Rank r's pages of the entries that requests give up, onto its stack in order.  The
// requests' entries, end to end, are dealt to the warps in equal shares: each counts
// its valid pages, the counts' sums say where it writes.  A cluster of `ctas` for a rank,
// each with a share of the requests.
constexpr int kReleaseRequests = 2048;  // requests whose entries are dealt at once
__global__ void __launch_bounds__(kThreadsPages) release_pages_kernel(const PageParams p, int ctas) {
    __shared__ int64_t warps[32];
    __shared__ int64_t off[kReleaseRequests + 1];
    __shared__ int low[kReleaseRequests];
    __shared__ GroupsHeld held;
    constexpr int kPer = kReleaseRequests / kThreadsPages;
    __shared__ Exchange exchange;
    const int r = blockIdx.x / ctas, cta = blockIdx.x - r * ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Groups groups = hold_groups(groups_of(p), &held);
    const int have = pages_free(p, r);
    int* free = p.free_pages + (int64_t)r * p.fp_sn;
    const int* row = p.bt + (int64_t)r * p.bt_sn;
    int64_t pushed = have;
    int turn = 0;
    const int per = min((p.B + ctas - 1) / ctas, kReleaseRequests);
    for (int64_t from = 0; from < p.B; from += (int64_t)per * ctas) {
        const int64_t b0 = from + (int64_t)cta * per;
        const int nb = (int)min(max(p.B - b0, (int64_t)0), (int64_t)per);
        int64_t sum = 0, mine[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int i = kPer * tid + e;
            const int64_t b = b0 + i;
            int count = 0;
            if (i < nb) {
                const int L = min(max(__ldg(p.lens + b), 0), p.max_seq_len);
                int keep = __ldg(p.keep_lens + b);
                keep = keep < 0 ? L : min(keep, L);
                low[i] = max(entries_of(p, keep, r), p.G ? member_of(groups, (int)b).entries : 0);
                count = max(entries_of(p, L, r) - low[i], 0);
                if (p.lens_out && r == 0) p.lens_out[b] = keep;
            }
            mine[e] = sum;
            sum += count;
        }
        int64_t total;
        const int64_t before = block_scan(sum, warps, &total) - sum;
#pragma unroll
        for (int e = 0; e < kPer; ++e) off[kPer * tid + e] = before + mine[e];
        __syncthreads();
        const int64_t share = ((total + kThreadsPages - 1) / kThreadsPages) * 32;  // entries of a warp
        const int64_t e0 = min(warp * share, total), e1 = min(e0 + share, total);
        // four steps' entries, -1 behind the last one; what they name is looked at when all are on their way
        auto pages_at = [&](int64_t e, int (&pg)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                pg[k] = -1;
                if (e + 32 * k >= e1) continue;  // the whole warp
                const int64_t at = min(e + 32 * k + lane, e1 - 1);
                const int i = last_at_or_before(off, nb, at);
                pg[k] = __ldg(row + (b0 + i) * p.bt_sb + low[i] + (at - off[i]));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (e + 32 * k + lane >= e1 || (unsigned)pg[k] >= (unsigned)p.num_pages) pg[k] = -1;
        };
        int64_t valid = 0;
        int pg[4];
        for (int64_t e = e0; e < e1; e += 128) {
            pages_at(e, pg);
#pragma unroll
            for (int k = 0; k < 4; ++k) valid += __popc(__ballot_sync(0xffffffffu, pg[k] >= 0));
        }
        const int64_t upto = block_scan(lane == 0 ? valid : 0, warps, &total);
        const int64_t others = sum_before(total, &exchange, ctas, turn++, &total);
        int64_t at = pushed + others + __shfl_sync(0xffffffffu, upto, 0) - valid;
        for (int64_t e = e0; e < e1; e += 128) {
            if (e1 - e0 > 128) pages_at(e, pg);  // (else they are still there)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned on = __ballot_sync(0xffffffffu, pg[k] >= 0);
                const int64_t to = at + __popc(on & ((1u << lane) - 1u));
                if (pg[k] >= 0 && to < p.free_capacity) free[to] = pg[k];
                at += __popc(on);
            }
        }
        pushed += total;
        __syncthreads();
    }
    __syncthreads();  // free_out may be free_count
    if (ctas > 1) sm100::cluster_sync();
    if (cta == 0 && tid == 0) p.free_out[r] = (int)min(pushed, (int64_t)p.free_capacity);
}

}  // namespace

namespace {

// A cluster of `ctas` for each of `clusters`.
template <class... A>
cudaError_t launch_clusters(void (*kernel)(A...), int clusters, int ctas, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)clusters * ctas);
    cfg.blockDim = dim3(kThreadsPages);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

cudaError_t launch_page_reserve(const PageParams& p, cudaStream_t stream) {
    // One launch instead of two while its eight CTAs are enough (64 requests: 15 us a call and 8.2 replayed,
    // a call with two 18).
    if ((int64_t)p.N * p.B <= 4096 && p.T <= 65536) return launch_clusters(reserve_small_kernel, 1, kCluster, stream, p);
    const cudaError_t e = launch_clusters(reserve_pages_kernel, p.N, p.B > 512 ? kCluster : 1, stream, p,
                                          p.B > 512 ? kCluster : 1);
    if (e != cudaSuccess) return e;
    const bool arrays = p.positions || p.slots || p.requests;
    if (!p.G && (!arrays || p.T == 0)) return cudaSuccess;
    const int64_t copies = p.G ? (int64_t)p.N * p.B * 32 : 0, tokens = arrays ? p.T : 0;
    const int64_t blocks = ((copies > tokens ? copies : tokens) + 255) / 256, most = 8ll * device_sm_count();
    return launch_chained(reserve_rest_kernel, (unsigned)(blocks < most ? blocks : most), 256, 0, stream, p);
}

cudaError_t launch_page_release(const PageParams& p, cudaStream_t stream) {
    // entries that a rank's requests may give up
    const int64_t cap = (((int64_t)p.max_seq_len + p.N - 1) / p.N + (1 << p.page_shift) - 1) >> p.page_shift;
    const int ctas = p.B > 512 || p.B * cap > 16384 ? kCluster : 1;
    return launch_clusters(release_pages_kernel, p.N, ctas, stream, p, ctas);
}

}  // namespace dcp
