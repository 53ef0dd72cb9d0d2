// dcp_evict.cu -- eviction by accumulated attention weight: per (rank, request,
// KV head) the K most attended tokens and the recent ones are kept, in order,
// and their K and V rows move to new pages.
//
// Selection: the weights become unsigned keys of the same order (NaN lowest);
// four passes over 8 bits each, a histogram in shared memory a pass, give the
// K-th largest key; one more pass lists the kept tokens by an ordered block
// scan, ties at the K-th key going to the lowest indices.  Nothing depends on
// the order of atomics.  The rows then move by a second kernel, whose bytes are
// the cost: two reads and two writes of every kept head row.
#include "dcp_chunk.cuh"

namespace dcp {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;

// Larger floats give larger keys; -0 and +0 the same; NaN 0.
__device__ __forceinline__ unsigned weight_key(float f) {
    if (!(f == f)) return 0u;
    unsigned u = __float_as_uint(f + 0.f);  // -0 becomes +0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams e) {
    const ChunkParams& p = e.c;
    __shared__ int hist[256];
    __shared__ int part[kSelWarps];
    __shared__ int found[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hkv = blockIdx.x % p.Hkv;
    const int rb = blockIdx.x / p.Hkv;
    const int b = rb % p.B, r = rb / p.B;
    const int keep_b = __ldg(e.keep_lens + b);
    if (keep_b < 0) return;
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len);
    const int held = rank_share(L, r, p.N);
    const int K = rank_share(min(L, min(keep_b, e.max_keep)), r, p.N);
    if (K == 0) return;
    const int older = rank_share(L - min(e.recent, L), r, p.N);  // tokens before the recent window
    const int want = K - (held - older);                        // of them are kept, by weight
    const float* acc = p.acc + (int64_t)r * p.a_sn + (int64_t)b * p.a_sb + (int64_t)hkv * p.a_sh;
    int* kept = e.kept + (int64_t)r * e.kp_sn + (int64_t)b * e.kp_sb + (int64_t)hkv * e.kp_sh;
    float* out = e.acc_out + (int64_t)r * e.ao_sn + (int64_t)b * e.ao_sb + (int64_t)hkv * e.ao_sh;
    if (want <= 0) {  // the latest K tokens
        for (int n = tid; n < K; n += kSelThreads) {
            kept[n] = held - K + n;
            out[n] = acc[held - K + n];
        }
        return;
    }
    // the want-th largest key, and how many of its equals are taken
    unsigned prefix = 0u, mask = 0u;
    int left = want;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < older; i += kSelThreads) {
            const unsigned k = weight_key(__ldg(acc + i));
            if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {  // lane l: bins 255 - 8 l down to 248 - 8 l
            int c[8], s = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) s += c[i] = hist[255 - 8 * lane - i];
            int up = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, up, o);
                if (lane >= o) up += x;
            }
            int above = up - s;
            if (above < left && up >= left) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (above < left && above + c[i] >= left) {
                        found[0] = 255 - 8 * lane - i;
                        found[1] = above;
                    }
                    above += c[i];
                }
            }
        }
        __syncthreads();
        prefix |= (unsigned)found[0] << shift;
        mask |= 255u << shift;
        left -= found[1];
        __syncthreads();
    }
    // the kept tokens in order; every thread counts the kept and the equal ones before it
    int base = 0, equal = 0;  // so far
    for (int i0 = 0; i0 < older; i0 += kSelThreads) {
        const int i = i0 + tid;
        const float a = i < older ? acc[i] : 0.f;
        const unsigned k = i < older ? weight_key(a) : 0u;
        const bool gt = i < older && k > prefix, eq = i < older && k == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) part[warp] = __popc(bg) | (__popc(be) << 16);
        __syncthreads();
        int g0 = 0, e0 = 0, gs = 0, es = 0;
#pragma unroll
        for (int w = 0; w < kSelWarps; ++w) {
            const int x = part[w];
            if (w < warp) {
                g0 += x & 0xffff;
                e0 += x >> 16;
            }
            gs += x & 0xffff;
            es += x >> 16;
        }
        const unsigned below = (1u << lane) - 1u;
        const int ne = equal + e0 + __popc(be & below);  // equal ones before this token
        const int ng = g0 + __popc(bg & below);
        if (gt || (eq && ne < left)) {
            const int n = base + ng + min(ne, left) - min(equal, left);
            kept[n] = i;
            out[n] = a;
        }
        base += gs + min(equal + es, left) - min(equal, left);
        equal += es;
        __syncthreads();
    }
    for (int n = want + tid; n < K; n += kSelThreads) {
        kept[n] = older + n - want;
        out[n] = acc[older + n - want];
    }
}

// Moves the kept head rows: 16 bytes a thread of one row, K and V.
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams e, int per_row, int blocks) {
    const ChunkParams& p = e.c;
    const int chunk = blockIdx.x % blocks;
    const int hkv = (blockIdx.x / blocks) % p.Hkv;
    const int rb = blockIdx.x / blocks / p.Hkv;
    const int b = rb % p.B, r = rb / p.B;
    const int keep_b = __ldg(e.keep_lens + b);
    if (keep_b < 0) return;
    const int L = min(max(__ldg(p.seq_lens + b), 0), p.max_seq_len);
    const int K = rank_share(min(L, min(keep_b, e.max_keep)), r, p.N);
    const int id = chunk * kMoveThreads + threadIdx.x;
    const int n = id / per_row, u = id % per_row;
    if (n >= K) return;
    const int src = e.kept[(int64_t)r * e.kp_sn + (int64_t)b * e.kp_sb + (int64_t)hkv * e.kp_sh + n];
    const int to = __ldg(e.dt + (int64_t)r * e.dt_sn + (int64_t)b * e.dt_sb + (n >> p.page_shift));
    if ((unsigned)to >= (unsigned)p.num_pages) return;
    const int from = page_of(p, r, b, src);
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (from >= 0) {
        k = *reinterpret_cast<const uint4*>(p.k + k_offset(p, r, from, src, hkv) + 16 * u);
        v = *reinterpret_cast<const uint4*>(p.v + v_offset(p, r, from, src, hkv) + 16 * u);
    }
    *reinterpret_cast<uint4*>(p.k + k_offset(p, r, to, n, hkv) + 16 * u) = k;
    *reinterpret_cast<uint4*>(p.v + v_offset(p, r, to, n, hkv) + 16 * u) = v;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& e, cudaStream_t stream) {
    const ChunkParams& p = e.c;
    const unsigned items = (unsigned)((int64_t)p.N * p.B * p.Hkv);
    evict_select_kernel<<<items, kSelThreads, 0, stream>>>(e);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    const int per_row = e.row_bytes / 16;
    const int64_t cap = ((int64_t)e.max_keep + p.N - 1) / p.N;
    const int64_t blocks = (cap * per_row + kMoveThreads - 1) / kMoveThreads;
    if (blocks == 0) return cudaSuccess;
    evict_move_kernel<<<(unsigned)(items * blocks), kMoveThreads, 0, stream>>>(e, per_row, (int)blocks);
    return cudaGetLastError();
}

}  // namespace dcp
