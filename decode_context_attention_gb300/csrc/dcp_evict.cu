// dcp_evict.cu -- eviction by accumulated attention weight: per (rank, request,
// KV head) the K most attended tokens and the recent ones are kept, in order,
// and their K and V rows move to new pages.
//
// Selection.  The weights become unsigned keys of the same order (NaN lowest);
// three passes over 11, 11 and 10 bits, a histogram each, give the K-th largest
// key, and one more lists the kept tokens by an ordered scan, ties at the K-th key
// going to the lowest indices.  Nothing depends on the order of atomics.  A
// problem is a cluster of 1 to 8 CTAs: each holds its slice of the keys in shared
// memory (read once), sums the histograms of all of them and takes its place in
// the order from the counts of those before it, through distributed shared
// memory.  What bounds it is the chain of passes and cluster barriers, not the
// bytes.
// The rows then move by a second kernel, whose bytes are the cost: two reads and
// two writes of every kept head row, four rows a thread in flight.
// Measured (bf16, D = 128): 32 requests of 8192 tokens on 4 ranks cut to half, 4 KV
// heads: 106 us, of which 84 move 537 MB (6.4 TB/s) and the rest selects;
// 131072 tokens to 8192 on 2 ranks, 8 KV heads: 43 us, 30 of them the selection.
#include <cooperative_groups.h>

#include "dcp_chunk.cuh"

namespace cg = cooperative_groups;

namespace dcp {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeld = 40 * 1024;  // keys of a CTA's slice that shared memory takes (160 KB); longer ones are read again
constexpr unsigned kAll = 0xffffffffu;

// Larger floats give larger keys; -0 and +0 the same; NaN 0.
__device__ __forceinline__ unsigned weight_key(float f) {
    if (!(f == f)) return 0u;
    const unsigned u = __float_as_uint(f + 0.f);  // -0 becomes +0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

struct SelectShared {
    // of alternate passes, so that a neighbour may still read the last one; read as int4
    alignas(16) int hist[2][kBins];
    int part[kSelWarps];
    int found, above;      // the bin of the K-th largest key, and how many keys lie above it
    int counts[2];         // keys of this slice above the K-th largest, and equal to it
};

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams e, int held_keys) {
    const ChunkParams& p = e.c;
    extern __shared__ unsigned keys_s[];
    __shared__ SelectShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = (int)cluster.num_blocks(), cr = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int problem = blockIdx.x / cs;
    const int hkv = problem % p.Hkv;
    const int rb = problem / p.Hkv;
    const int b = rb % p.B, r = rb / p.B;
    // the whole cluster leaves together
    const int keep_b = __ldg(e.keep_lens + b);
    if (keep_b < 0) return;
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len);
    const int held = rank_share(L, r, p.N);
    const int K = rank_share(min(L, min(keep_b, e.max_keep)), r, p.N);
    if (K == 0) return;
    const int older = rank_share(L - min(e.recent, L), r, p.N);  // tokens before the recent window
    const int want = max(K - (held - older), 0);                // of them are kept, by weight
    const float* acc = p.acc + (int64_t)r * p.a_sn + (int64_t)b * p.a_sb + (int64_t)hkv * p.a_sh;
    int* kept = e.kept + (int64_t)r * e.kp_sn + (int64_t)b * e.kp_sb + (int64_t)hkv * e.kp_sh;
    float* out = e.acc_out + (int64_t)r * e.ao_sn + (int64_t)b * e.ao_sb + (int64_t)hkv * e.ao_sh;
    // the window's tokens (the latest of them when it holds more than is kept) follow the older ones
    for (int n = want + cr * kSelThreads + tid; n < K; n += cs * kSelThreads) {
        const int i = held - K + n;
        kept[n] = i;
        out[n] = acc[i];
    }
    if (want == 0) return;
    // this CTA's slice [lo, hi), a whole number of steps of four keys a thread
    constexpr int kStep = 4 * kSelThreads;
    const int steps = (older + kStep - 1) / kStep;
    const int per = (steps + cs - 1) / cs;
    const int lo = min(cr * per * kStep, older), hi = min(lo + per * kStep, older);
    const bool in_smem = hi - lo <= held_keys;
    for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
    // the want-th largest key, and how many of its equals are taken
    unsigned prefix = 0u, mask = 0u;
    int left = want;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const unsigned bins = pass == 2 ? 1023u : 2047u;
        int* hist = sh.hist[pass & 1];
        for (int i = lo + tid; i < hi; i += kSelThreads) {
            unsigned k;
            if (pass == 0 || !in_smem) {
                k = weight_key(__ldg(acc + i));
                if (pass == 0 && in_smem) keys_s[i - lo] = k;
            } else {
                k = keys_s[i - lo];
            }
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & bins], 1);
        }
        if (cs > 1) cluster.sync();
        else __syncthreads();
        // thread t: bins top - 4 t down to top - 4 t - 3, over the whole cluster
        int c[4] = {0, 0, 0, 0};
        const int top = (int)bins - 4 * tid;
        if (top >= 3) {
            for (int q = 0; q < cs; ++q) {
                const int4 v = *reinterpret_cast<const int4*>(
                    (cs > 1 ? cluster.map_shared_rank(hist, q) : hist) + top - 3);
                c[0] += v.w;
                c[1] += v.z;
                c[2] += v.y;
                c[3] += v.x;
            }
        }
        const int s = c[0] + c[1] + c[2] + c[3];
        int up = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kAll, up, o);
            if (lane >= o) up += x;
        }
        if (lane == 31) sh.part[warp] = up;
        __syncthreads();
        for (int w = 0; w < warp; ++w) up += sh.part[w];
        int above = up - s;
        if (above < left && up >= left) {  // one thread of the CTA
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (above < left && above + c[i] >= left) {
                    sh.found = top - i;
                    sh.above = above;
                }
                above += c[i];
            }
        }
        __syncthreads();
        prefix |= (unsigned)sh.found << shift;
        mask |= bins << shift;
        left -= sh.above;
        if (pass == 0) {  // the first histogram is used again by the last pass, once every neighbour has read it
            if (cs > 1) cluster.sync();
            for (int i = tid; i < kBins; i += kSelThreads) sh.hist[0][i] = 0;
        }
        __syncthreads();
    }
    // how many of this slice's keys are above the K-th largest, and equal to it
    {
        int g = 0, q = 0;
        for (int i = lo + tid; i < hi; i += kSelThreads) {
            const unsigned k = in_smem ? keys_s[i - lo] : weight_key(__ldg(acc + i));
            g += k > prefix;
            q += k == prefix;
        }
        g = __reduce_add_sync(kAll, g);
        q = __reduce_add_sync(kAll, q);
        if (tid < 2) sh.counts[tid] = 0;
        __syncthreads();
        if (lane == 0) {
            atomicAdd(&sh.counts[0], g);
            atomicAdd(&sh.counts[1], q);
        }
    }
    int base = 0, equal = 0;  // kept ones and equal ones before this slice
    if (cs > 1) {
        cluster.sync();
        for (int q = 0; q < cr; ++q) {
            const int* c = cluster.map_shared_rank(sh.counts, q);
            base += c[0];
            equal += c[1];
        }
        cluster.sync();  // no CTA ends while another may read its shared memory
    }
    base += min(equal, left);
    // the kept tokens in order: four neighbouring keys a thread and step
    for (int i0 = lo; i0 < hi; i0 += kStep) {
        const int i = i0 + 4 * tid;
        unsigned k[4];
        int gt = 0, eq = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const bool ok = i + x < hi;
            k[x] = !ok ? 0u : in_smem ? keys_s[i + x - lo] : weight_key(__ldg(acc + i + x));
            gt += ok && k[x] > prefix;
            eq += ok && k[x] == prefix;
        }
        int up = gt | (eq << 16);  // both below 2^16 over a step
        const int mine = up;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kAll, up, o);
            if (lane >= o) up += x;
        }
        if (lane == 31) sh.part[warp] = up;
        __syncthreads();
        int before = up - mine, all = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) before += sh.part[w];
            all += sh.part[w];
        }
        int ng = before & 0xffff, ne = equal + (before >> 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (i + x >= hi) break;
            const bool is_gt = k[x] > prefix, is_eq = k[x] == prefix;
            if (is_gt || (is_eq && ne < left)) {
                const int n = base + ng + min(ne, left) - min(equal, left);
                kept[n] = i + x;
                out[n] = __ldg(acc + i + x);
            }
            ng += is_gt;
            ne += is_eq;
        }
        const int step_eq = all >> 16;
        base += (all & 0xffff) + min(equal + step_eq, left) - min(equal, left);
        equal += step_eq;
        __syncthreads();
    }
}

// Moves the kept head rows: a thread has 16 bytes of four rows, K and V.
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams e, int per_row, int blocks) {
    const ChunkParams& p = e.c;
    const int chunk = blockIdx.x % blocks;
    const int hkv = (blockIdx.x / blocks) % p.Hkv;
    const int rb = blockIdx.x / blocks / p.Hkv;
    const int b = rb % p.B, r = rb / p.B;
    const int rows = kMoveThreads / per_row;  // rows of a step; threads past rows * per_row have none
    const int row = threadIdx.x / per_row, u = threadIdx.x - row * per_row;
    const int n0 = chunk * rows * kMoveRows + row;
    const int keep_b = __ldg(e.keep_lens + b);
    if (keep_b < 0 || row >= rows) return;
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len);
    const int K = rank_share(min(L, min(keep_b, e.max_keep)), r, p.N);
    const int* kept = e.kept + (int64_t)r * e.kp_sn + (int64_t)b * e.kp_sb + (int64_t)hkv * e.kp_sh;
    int src[kMoveRows], to[kMoveRows], from[kMoveRows];
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
        const int n = n0 + x * rows;
        src[x] = n < K ? kept[n] : 0;
        to[x] = n < K ? __ldg(e.dt + (int64_t)r * e.dt_sn + (int64_t)b * e.dt_sb + (n >> p.page_shift)) : -1;
    }
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) from[x] = n0 + x * rows < K ? page_of(p, r, b, src[x]) : -1;
    uint4 k[kMoveRows], v[kMoveRows];
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
        k[x] = v[x] = make_uint4(0u, 0u, 0u, 0u);
        if (from[x] >= 0) {
            k[x] = __ldcs(reinterpret_cast<const uint4*>(p.k + k_offset(p, r, from[x], src[x], hkv) + 16 * u));
            v[x] = __ldcs(reinterpret_cast<const uint4*>(p.v + v_offset(p, r, from[x], src[x], hkv) + 16 * u));
        }
    }
#pragma unroll
    for (int x = 0; x < kMoveRows; ++x) {
        if ((unsigned)to[x] >= (unsigned)p.num_pages) continue;
        const int n = n0 + x * rows;
        *reinterpret_cast<uint4*>(p.k + k_offset(p, r, to[x], n, hkv) + 16 * u) = k[x];
        *reinterpret_cast<uint4*>(p.v + v_offset(p, r, to[x], n, hkv) + 16 * u) = v[x];
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& e, cudaStream_t stream) {
    const ChunkParams& p = e.c;
    const int64_t problems = (int64_t)p.N * p.B * p.Hkv;
    const int64_t cap = ((int64_t)p.max_seq_len + p.N - 1) / p.N;
    // CTAs of a problem: as many as the SMs have room for, a step of keys each at
    // least (131072 tokens, 16 problems: 43 us with 8, 151 us with one; 512 problems
    // fill the SMs with one each: 106 us)
    int cs = 1;
    while (cs < 8 && problems * cs * 2 <= 2 * device_sm_count() && cap > (int64_t)cs * 4 * kSelThreads) cs *= 2;
    const int64_t slice = (((cap + 4 * kSelThreads - 1) / (4 * kSelThreads) + cs - 1) / cs) * 4 * kSelThreads;
    const int held = (int)(slice < kHeld ? slice : kHeld);
    cudaError_t err =
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(problems * cs));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)held * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, evict_select_kernel, e, held);
    if (err != cudaSuccess) return err;
    const int per_row = e.row_bytes / 16;  // at most 128
    const int64_t kcap = ((int64_t)e.max_keep + p.N - 1) / p.N;
    const int64_t rows = (int64_t)(kMoveThreads / per_row) * kMoveRows;
    const int64_t blocks = (kcap + rows - 1) / rows;
    if (blocks == 0) return cudaSuccess;
    evict_move_kernel<<<(unsigned)(problems * blocks), kMoveThreads, 0, stream>>>(e, per_row, (int)blocks);
    return cudaGetLastError();
}

}  // namespace dcp
