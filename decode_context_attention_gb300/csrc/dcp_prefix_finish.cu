// dcp_prefix_finish.cu -- the last step of the attention of a batch that shares
// prefixes: requests' own parts of few rows and tokens, and the join of every
// request's common and own parts.
//
// Joining parts over disjoint tokens with outputs o_i and log-sum-exps z_i:
//     z = log2 sum_i 2^z_i,  o = sum_i 2^(z_i - z) o_i.
//
// An own part of a decode step is a few rows (new tokens x heads of a group) over some
// hundred tokens: 100 to 300 KB of keys and values and hardly any arithmetic.  One CTA
// of four warps takes one (request, rank, KV head), a warp 16 rows at a time over every
// fourth (second, or every) tile of 16 tokens.  Keys and values go from memory into the
// registers of mma.sync's (m16n8k16) operands without a stop: the order of the elements
// of a head's row along the products' sums is free as long as both operands have the
// same one, so lane (g, c) takes 16 adjacent bytes of token g's key, eights of a 64-byte
// group; and the order of the output's columns is free, so it takes 16 adjacent bytes of
// four tokens' values and pairs them up by byte permutes.  What bounds it is the bytes in flight: a
// warp has a tile's values under way while the scores are computed and the next tile's
// keys while the value product is.
// One pass, an online softmax with the reference maximum moved when it is passed by 2^8,
// as in the tensor-core kernel.
#include <type_traits>

#include "dcp_chunk.cuh"
#include "dcp_mma.cuh"

namespace dcp {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kFinishThreads = 128;
constexpr int kMaxRanges = 512;  // CTAs of the kernel before
constexpr int kJoinRows = 4;     // rows of a warp

// A row's weights are 2^(s - m + kBias): fp16's smallest normal is 2^-14, and a largest
// weight of up to 2^15 keeps those of a long tail (dcp_chunk_attention_tc.cu).
constexpr float kGrow = 8.f;
template <typename T>
constexpr float kBias = std::is_same<T, __half>::value ? 7.f : 0.f;

template <int D>
struct Slim {
    static constexpr int WD = D == 256 ? 2 : 1;       // warps that share a tile's columns
    static constexpr int WX = 4 / WD;                 // warps for row blocks and token tiles
    static constexpr int DW = D / WD;                 // columns of a warp
    static constexpr int kRows = 16 * WX;             // rows of an item, at most
    static constexpr int kPitch = D * 2 + 64;         // bytes of a staged query row: no bank conflicts
    static constexpr int kSmemQ = kRows * kPitch, kSmemO = WX * 16 * D * 4;
    static constexpr int kSmem = kSmemQ > kSmemO ? kSmemQ : kSmemO;
};

// Where the parts of a common item lie: slots of the chunk kernel's partials, or (n = -1) the plan's rows.
struct Parts {
    int n;
    int slot[kMaxRanges + 1];
};

// The parts of the item, by one warp.
__device__ void find_parts(const ChunkPos* pos, int ctas, const ChunkPos& item, Parts* parts) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int k = lane; k <= ctas; k += 32) {
        const ChunkPos x = pos[k];
        before += (x.b != item.b     ? x.b < item.b
                   : x.rh != item.rh ? x.rh < item.rh
                   : x.qt != item.qt ? x.qt < item.qt
                                     : x.tile == 0)
                      ? 1
                      : 0;
    }
    const int c = (int)__reduce_add_sync(kAll, (unsigned)before) - 1;  // the range with the item's first tile
    if (c < 0 || c >= ctas || !same_item(pos[c + 1], item)) {
        if (lane == 0) parts->n = -1;
        return;
    }
    if (lane == 0) parts->slot[0] = 2 * c + (same_item(pos[c], item) ? 0 : 1);
    int n = 1;
    for (int k0 = c + 1;; k0 += 32) {
        const int k = k0 + lane;
        const ChunkPos x = pos[min(k, ctas)], y = pos[min(k + 1, ctas)];
        const bool in = k < ctas && same_item(x, item);
        // a range that lies empty inside the item left nothing
        const unsigned on = __ballot_sync(kAll, in && !(same_item(y, item) && y.tile == x.tile));
        if (on >> lane & 1) parts->slot[n + __popc(on & ((1u << lane) - 1u))] = 2 * k;
        n += __popc(on);
        if (!__all_sync(kAll, in)) break;
    }
    if (lane == 0) parts->n = n;
}

// The joined row so far: base-2 log-sum-exp of the largest part, sum of the weights, and
// this lane's share of the outputs.
template <int NV>
struct Joined {
    float mx, sum;
    float4 acc[NV];
};
template <int NV>
__device__ __forceinline__ void join2(Joined<NV>& a, float z0, const float4 (&o0)[NV], float z1, const float4 (&o1)[NV]) {
    // mx becomes finite, infinite or NaN with the parts: as the formula has it
    const float m = fmaxf(a.mx, fmaxf(z0, z1));
    const float old = a.mx == -INFINITY ? 0.f : exp2f(a.mx - m);
    const float w0 = z0 == -INFINITY ? 0.f : exp2f(z0 - m), w1 = z1 == -INFINITY ? 0.f : exp2f(z1 - m);
    a.mx = m;
    a.sum = fmaf(a.sum, old, w0 + w1);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        a.acc[v].x = fmaf(w1, o1[v].x, fmaf(w0, o0[v].x, a.acc[v].x * old));
        a.acc[v].y = fmaf(w1, o1[v].y, fmaf(w0, o0[v].y, a.acc[v].y * old));
        a.acc[v].z = fmaf(w1, o1[v].z, fmaf(w0, o0[v].z, a.acc[v].z * old));
        a.acc[v].w = fmaf(w1, o1[v].w, fmaf(w0, o0[v].w, a.acc[v].w * old));
    }
}
template <typename T, int D, int NV>
__device__ __forceinline__ void write_row(const PrefixParams& p, int r, int64_t t, int h, const Joined<NV>& a) {
    const int lane = threadIdx.x & 31;
    const float inv = a.sum == 0.f ? 0.f : 1.f / a.sum;
    unsigned char* out = p.o + (int64_t)r * p.o_sn + t * p.o_st + (int64_t)h * p.o_sh;
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (4 * lane + 128 * v < D) {
            const float4 x = a.acc[v];
            *reinterpret_cast<uint2*>(out + 2 * (4 * lane + 128 * v)) =
                make_uint2(f32_to_pair(make_float2(x.x * inv, x.y * inv), T()),
                           f32_to_pair(make_float2(x.z * inv, x.w * inv), T()));
        }
    if (lane == 0) {
        const float lse2 = a.sum == 0.f ? -INFINITY : a.mx + log2f(a.sum);
        p.lse[(int64_t)r * p.l_sn + t * p.l_st + (int64_t)h * p.l_sh] = p.base2 ? lse2 : lse2 * kLn2;
    }
}

// ---------------------------------------------------------------------------
// slim own parts
// ---------------------------------------------------------------------------

template <typename T, int D>
__device__ void slim_part(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int64_t item,
                          unsigned char* smem) {
    using S = Slim<D>;
    constexpr int WX = S::WX, DW = S::DW, NV = (D + 127) / 128;
    constexpr int KC = D / 32, VC = DW / 64;  // 16-byte pieces of a key and a value row that a lane takes
    __shared__ float row_m[WX * 16], row_l[WX * 16];
    __shared__ unsigned poison[4];  // tokens of the masked tiles whose V row is not finite
    __shared__ Parts parts[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int hkv = (int)(item % p.Hkv), r = (int)(item / p.Hkv % p.N), b = (int)(item / p.Hkv / p.N);
    const Planned q = load_planned(p.slim + 2 * (int64_t)b);
    if (q.n == 0) return;
    const int nrows = q.n * p.gq;
    const int lim0 = visible(p, q, 0, r), lim_last = visible(p, q, q.n - 1, r);
    const int64_t table = table_at(p, q, r, b);
    // row blocks, and tiles between them
    const int wr = nrows <= 16 ? 1 : nrows <= 32 ? 2 : 4, wt = WX / wr;
    const int wd = warp / WX, wx = warp % WX, blk = wx % wr, first = wx / wr;
    for (int id = tid; id < 16 * wr * (D / 8); id += kFinishThreads) {
        const int row = id / (D / 8), u = id % (D / 8);
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (row < nrows)
            x = __ldg(reinterpret_cast<const uint4*>(p.q + (int64_t)(q.start + row / p.gq) * p.q_st +
                                                     (int64_t)(hkv * p.gq + row % p.gq) * p.q_sh) + u);
        *reinterpret_cast<uint4*>(smem + row * S::kPitch + 16 * u) = x;
    }
    if (tid < 4) poison[tid] = 0u;
    // scores enter with the scale's sign, so that the maximum is that of the scaled ones
    const float sign = p.sm_scale < 0.f ? -1.f : 1.f, qs = fabsf(p.sm_scale) * kLog2e;
    int lim[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * blk + g + 8 * i;
        lim[i] = row < nrows ? visible(p, q, row / p.gq, r) : 0;
    }
    const unsigned char* kbase = p.k + (int64_t)r * p.k_sn + (int64_t)hkv * p.k_sh + 16 * c;
    const unsigned char* vbase = p.v + (int64_t)r * p.v_sn + (int64_t)hkv * p.v_sh + 2 * DW * wd + 16 * g;
    const int mask = (1 << p.page_shift) - 1;
    // page of the tile's token lane % 16, -1 behind the last one and outside of the pool
    auto page_at = [&](int t) -> int {
        const int i = t + (lane & 15);
        return i < lim_last ? page_in(p, table, i) : -1;
    };
    uint4 k[2][KC], v[4][VC];
    auto load_k = [&](int t, int pages) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = g + 8 * e, pg = __shfl_sync(kAll, pages, i);
            const unsigned char* at = kbase + (int64_t)pg * p.k_sp + (int64_t)((t + i) & mask) * p.k_st;
#pragma unroll
            for (int x = 0; x < KC; ++x)
                k[e][x] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(at + 64 * x)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto load_v = [&](int t, int pages) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 2 * c + (e & 1) + 8 * (e >> 1), pg = __shfl_sync(kAll, pages, i);
            const unsigned char* at = vbase + (int64_t)pg * p.v_sp + (int64_t)((t + i) & mask) * p.v_st;
#pragma unroll
            for (int x = 0; x < VC; ++x)
                v[e][x] = pg >= 0 ? __ldg(reinterpret_cast<const uint4*>(at + 128 * x)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    float o[8 * VC][4];
#pragma unroll
    for (int i = 0; i < 8 * VC; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int t = 16 * first, pages = page_at(t);
    if (t < lim_last) load_k(t, pages);
    __syncthreads();
    const unsigned char* qa = smem + (16 * blk + g) * S::kPitch + 16 * c;
    while (t < lim_last) {
        load_v(t, pages);
        const int next = t + 16 * wt;
        const int pages_next = page_at(next);
        float s[2][4] = {};
#pragma unroll
        for (int x = 0; x < KC; ++x) {
            const uint4 a = *reinterpret_cast<const uint4*>(qa + 64 * x);
            const uint4 a8 = *reinterpret_cast<const uint4*>(qa + 8 * S::kPitch + 64 * x);
            const unsigned lo[4] = {a.x, a8.x, a.y, a8.y}, hi[4] = {a.z, a8.z, a.w, a8.w};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mma16816<T>(s[e], lo, k[e][x].x, k[e][x].y);
                mma16816<T>(s[e], hi, k[e][x].z, k[e][x].w);
            }
        }
        if (next < lim_last) load_k(next, pages_next);
        const bool masked = t + 16 > lim0;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[e][x] *= sign;
                if (masked && t + 8 * e + 2 * c + (x & 1) >= lim[x >> 1]) s[e][x] = -INFINITY;
            }
        float mx[2];
        bool grow = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (a maximum over a lane's scores first: no lane of a row sees it grow unless the row does)
            mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            grow |= (mx[i] - ref[i]) * qs > kGrow || (ref[i] == -INFINITY && mx[i] > -INFINITY);
        }
        if (__any_sync(kAll, grow)) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kAll, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(kAll, mx[i], 2));
                // a row moves by its own maximum alone: rows of no query have no say in how others are rounded
                float alpha = 1.f;
                if ((mx[i] - ref[i]) * qs > kGrow || (ref[i] == -INFINITY && mx[i] > -INFINITY)) {
                    alpha = ref[i] == -INFINITY ? 0.f : exp2_fast((ref[i] - mx[i]) * qs);
                    ref[i] = mx[i];
                }
                l[i] *= alpha;
#pragma unroll
                for (int n = 0; n < 8 * VC; ++n) {
                    o[n][2 * i] *= alpha;
                    o[n][2 * i + 1] *= alpha;
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float m = ref[x >> 1];
                s[e][x] = s[e][x] == -INFINITY
                              ? 0.f  // (a scale of 0 times -infinity is no weight)
                              : exp2_fast(fmaf(s[e][x] - (m == -INFINITY ? 0.f : m), qs, kBias<T>));
                l[x >> 1] += s[e][x];
            }
        if (masked && lim0 < lim_last) {
            // a value that some rows may not see must not reach them as 0 * inf
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bool bad = false;
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                    uint4& w = v[e][x];
                    bad |= pair_nonfinite<T>(w.x) || pair_nonfinite<T>(w.y) || pair_nonfinite<T>(w.z) ||
                           pair_nonfinite<T>(w.w);
                    w = make_uint4(pair_finite<T>(w.x), pair_finite<T>(w.y), pair_finite<T>(w.z), pair_finite<T>(w.w));
                }
                // below 96, as an item's rows are at most 64 tokens' and what they see differs by less
                const int at = t - (lim0 & ~15) + 2 * c + (e & 1) + 8 * (e >> 1);
                if (bad && at < 128) atomicOr(&poison[at >> 5], 1u << (at & 31));
            }
        }
        // weights in the payload type (half a step a term); the row sums take them unrounded
        const unsigned a[4] = {f32_to_pair(make_float2(s[0][0], s[0][1]), T()),
                               f32_to_pair(make_float2(s[0][2], s[0][3]), T()),
                               f32_to_pair(make_float2(s[1][0], s[1][1]), T()),
                               f32_to_pair(make_float2(s[1][2], s[1][3]), T())};
#pragma unroll
        for (int x = 0; x < VC; ++x) {
            auto word = [](const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; };
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const unsigned sel = j & 1 ? 0x7632u : 0x5410u;
                mma16816<T>(o[8 * x + j], a, __byte_perm(word(v[0][x], j >> 1), word(v[1][x], j >> 1), sel),
                            __byte_perm(word(v[2][x], j >> 1), word(v[3][x], j >> 1), sel));
            }
        }
        t = next;
        pages = pages_next;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
    }
    __syncthreads();  // every warp is done with the queries
    float* os = reinterpret_cast<float*>(smem);  // [WX][16][D]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = 16 * wx + g + 8 * i;
        if (wd == 0 && c == 0) {
            row_m[at] = ref[i];
            row_l[at] = l[i];
        }
        // lane (g, c) holds columns 64 x + 16 c + [0, 16) of its warp's
#pragma unroll
        for (int x = 0; x < VC; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = 4 * (y & 1), z = 2 * i + (y >> 1);
                *reinterpret_cast<float4*>(os + (int64_t)at * D + DW * wd + 64 * x + 16 * c + 4 * y) =
                    make_float4(o[8 * x + j][z], o[8 * x + j + 1][z], o[8 * x + j + 2][z], o[8 * x + j + 3][z]);
            }
    }
    __syncthreads();
    // the warps' shares of a row (wt of them, 16 * wr rows apart) into the first one's place, normalised
    for (int row = warp; row < nrows; row += 4) {
        float m = -INFINITY;
        for (int x = 0; x < wt; ++x) m = fmaxf(m, row_m[row + 16 * wr * x]);
        const float base = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
        float4 acc[NV];
#pragma unroll
        for (int y = 0; y < NV; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < wt; ++x) {
            const int at = row + 16 * wr * x;
            const float w = row_m[at] == -INFINITY ? 0.f : exp2f((row_m[at] - base) * qs);
            // a share that has seen nothing is zero, and stays NaN where a score was
            sum = row_m[at] == -INFINITY ? sum + row_l[at] : fmaf(w, row_l[at], sum);
#pragma unroll
            for (int y = 0; y < NV; ++y)
                if (4 * lane + 128 * y < D) {
                    const float4 z = *reinterpret_cast<const float4*>(os + (int64_t)at * D + 4 * lane + 128 * y);
                    const float f = row_m[at] == -INFINITY ? 1.f : w;
                    acc[y].x = fmaf(f, z.x, acc[y].x);
                    acc[y].y = fmaf(f, z.y, acc[y].y);
                    acc[y].z = fmaf(f, z.z, acc[y].z);
                    acc[y].w = fmaf(f, z.w, acc[y].w);
                }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int y = 0; y < NV; ++y)
            if (4 * lane + 128 * y < D)
                *reinterpret_cast<float4*>(os + (int64_t)row * D + 4 * lane + 128 * y) =
                    make_float4(acc[y].x * inv, acc[y].y * inv, acc[y].z * inv, acc[y].w * inv);
        __syncwarp();
        if (lane == 0) row_l[row] = sum == 0.f ? -INFINITY : fmaf(m, qs, log2f(sum) - kBias<T>);
    }
    __syncthreads();
    if ((poison[0] | poison[1] | poison[2] | poison[3]) != 0u) {
        if (tid < nrows) {
            const T* qrow = reinterpret_cast<const T*>(p.q + (int64_t)(q.start + tid / p.gq) * p.q_st +
                                                       (int64_t)(hkv * p.gq + tid % p.gq) * p.q_sh);
            add_nonfinite<T, float>(p, r, table, hkv, qrow, lim0 & ~15, poison, 4, visible(p, q, tid / p.gq, r),
                                    row_l[tid], os + (int64_t)tid * D);
        }
        __syncthreads();
    }
    // what follows reads what the chunk kernel left
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool joined = q.kind == kOwn;
    int qt0 = 0, cstart = 0;
    if (joined) {
        const Planned common = load_request(p, q.common);
        cstart = common.start;
        joined = q.start >= cstart && q.start + q.n <= cstart + common.n;  // (groups out of order)
    }
    if (joined) {
        qt0 = (q.start - cstart) / tpi;
        const int last = (q.start + q.n - 1 - cstart) / tpi;
        if (warp < 2 && qt0 + warp <= last) {
            const ChunkPos x = {q.common, r * p.Hkv + hkv, qt0 + warp, 0};
            find_parts(ws.pos, ctas, x, &parts[warp]);
        }
        __syncthreads();
    }
    for (int row0 = kJoinRows * warp; row0 < nrows; row0 += 4 * kJoinRows) {
        Joined<NV> a[kJoinRows];
        int n[kJoinRows], most = 0;
        const Parts* from[kJoinRows];
        int64_t whole[kJoinRows], within[kJoinRows];
#pragma unroll
        for (int e = 0; e < kJoinRows; ++e) {
            const int row = min(row0 + e, nrows - 1), tok = q.start + row / p.gq, h = hkv * p.gq + row % p.gq;
            a[e].mx = row_l[row];
            a[e].sum = a[e].mx == -INFINITY ? 0.f : 1.f;
#pragma unroll
            for (int y = 0; y < NV; ++y)
                a[e].acc[y] = 4 * lane + 128 * y < D
                                  ? *reinterpret_cast<const float4*>(os + (int64_t)row * D + 4 * lane + 128 * y)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            const int qt = joined ? (tok - cstart) / tpi : 0;
            from[e] = &parts[qt - qt0 > 0 ? 1 : 0];
            n[e] = !joined ? 0 : from[e]->n < 0 ? 1 : from[e]->n;
            most = max(most, n[e]);
            whole[e] = (((int64_t)r) * p.T + tok) * p.H + h;
            within[e] = (int64_t)(tok - cstart - qt * tpi) * p.gq + row % p.gq;
        }
        // two parts at a time, all their rows in flight
        for (int i = 0; i < most; i += 2) {
            float z[kJoinRows][2];
            float4 x[kJoinRows][2][NV];
#pragma unroll
            for (int e = 0; e < kJoinRows; ++e)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const bool ok = i + y < n[e];
                    const bool cut = ok && from[e]->n >= 0;
                    const int64_t at = cut ? (int64_t)from[e]->slot[i + y] * rows + within[e] : whole[e];
                    z[e][y] = ok ? (cut ? ws.lse : p.wl)[at] : -INFINITY;
#pragma unroll
                    for (int w = 0; w < NV; ++w)
                        x[e][y][w] = ok && 4 * lane + 128 * w < D
                                         ? *reinterpret_cast<const float4*>((cut ? ws.o : p.wo) + at * D + 4 * lane + 128 * w)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int e = 0; e < kJoinRows; ++e) join2<NV>(a[e], z[e][0], x[e][0], z[e][1], x[e][1]);
        }
#pragma unroll
        for (int e = 0; e < kJoinRows; ++e) {
            const int row = row0 + e;
            if (row < nrows)
                write_row<T, D, NV>(p, r, q.start + row / p.gq, hkv * p.gq + row % p.gq, a[e]);
        }
    }
}

// ---------------------------------------------------------------------------
// the join of the parts that the chunk kernel has computed
// ---------------------------------------------------------------------------

// Rows of a part: their fp32 outputs and base-2 log-sum-exps, one after the other.
struct Rows {
    const float* o;
    const float* l;
};

template <typename T, int D>
__device__ void join_rest(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int worker,
                          int workers, unsigned char* smem) {
    constexpr int NV = (D + 127) / 128;  // 16-byte vectors of a lane
    constexpr int kWarps = kFinishThreads / 32;
    const int lane = threadIdx.x & 31;
    // the next kernel of the stream waits for this one only: it must not end before the chunk kernel has
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool wide = false;
    for (int k = threadIdx.x; k < p.plan_ctas; k += kFinishThreads) wide |= __ldg(p.wide + k) != 0;
    if (!__syncthreads_or(wide)) return;
    ChunkPos* pos = reinterpret_cast<ChunkPos*>(smem);
    for (int c = threadIdx.x; c <= ctas; c += kFinishThreads) pos[c] = ws.pos[c];
    __syncthreads();
    const int quads = (p.gq + kJoinRows - 1) / kJoinRows;
    const int tokens = min(max(__ldg(p.query_start + p.requests), 0), p.T);
    const int64_t tasks = (int64_t)tokens * p.N * p.Hkv * quads;
    for (int64_t task = (int64_t)worker * kWarps + (threadIdx.x >> 5); task < tasks; task += (int64_t)workers * kWarps) {
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
        if (t < own.start || t >= own.start + own.n) continue;  // a slim part's, or of no request
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
            c = (int)__reduce_add_sync(kAll, (unsigned)n) - 1;
            cut = c >= 0 && c < ctas && same_item(pos[c + 1], item);
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
        Joined<NV> a[kJoinRows];
#pragma unroll
        for (int e = 0; e < kJoinRows; ++e) {
            a[e].mx = -INFINITY;
            a[e].sum = 0.f;
#pragma unroll
            for (int y = 0; y < NV; ++y) a[e].acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        // two parts at a time, all their rows in flight
        for (Rows x[2] = {next(), next()}; x[0].o; x[0] = next(), x[1] = next()) {
            float z[kJoinRows][2];
            float4 o[kJoinRows][2][NV];
#pragma unroll
            for (int e = 0; e < kJoinRows; ++e)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const bool ok = x[y].o && e < nrows;
                    z[e][y] = ok ? x[y].l[e] : -INFINITY;
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        o[e][y][v] = ok && 4 * lane + 128 * v < D
                                         ? *reinterpret_cast<const float4*>(x[y].o + e * D + 4 * lane + 128 * v)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
            for (int e = 0; e < kJoinRows; ++e) join2<NV>(a[e], z[e][0], o[e][0], z[e][1], o[e][1]);
        }
#pragma unroll
        for (int e = 0; e < kJoinRows; ++e)
            if (e < nrows) write_row<T, D, NV>(p, r, t, hkv * p.gq + h0 + e, a[e]);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFinishThreads, D == 64 ? 4 : D == 128 ? 3 : 2)
    prefix_finish_kernel(const PrefixParams p, const ChunkPartials ws, int tpi, int rows, int ctas, int items) {
    extern __shared__ __align__(16) unsigned char smem[];
    if ((int)blockIdx.x < items)
        slim_part<T, D>(p, ws, tpi, rows, ctas, blockIdx.x, smem);
    else
        join_rest<T, D>(p, ws, tpi, rows, ctas, blockIdx.x - items, gridDim.x - items, smem);
}

template <typename T, int D>
cudaError_t launch(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, cudaStream_t stream) {
    const auto kernel = prefix_finish_kernel<T, D>;
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv;
    const int64_t tasks = (int64_t)p.T * p.N * p.Hkv * ((p.gq + kJoinRows - 1) / kJoinRows);
    const int64_t need = (tasks + kFinishThreads / 32 - 1) / (kFinishThreads / 32), most = 4ll * device_sm_count();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items + (need < most ? need : most)));
    cfg.blockDim = dim3(kFinishThreads);
    cfg.dynamicSmemBytes = Slim<D>::kSmem;
    cfg.stream = stream;
    // the chunk kernel lets this one start as soon as an SM is free of it: slim parts need nothing of its results
    // until their join (griddepcontrol.wait)
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, ws, tpi, rows, ctas, (int)items);
}

template <typename T>
cudaError_t launch_d(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, cudaStream_t stream) {
    switch (p.D) {
        case 64: return launch<T, 64>(p, ws, tpi, rows, ctas, stream);
        case 128: return launch<T, 128>(p, ws, tpi, rows, ctas, stream);
        case 256: return launch<T, 256>(p, ws, tpi, rows, ctas, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// An own part is slim up to the rows of a CTA, and up to as many tokens of a rank as
// keep its one CTA from outlasting the others: with fewer parts than CTAs fit at once, a
// long part is better cut over the SMs.
void slim_limits(PrefixParams& p) {
    p.slim_rows = p.D == 256 ? Slim<256>::kRows : Slim<128>::kRows;
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv, slots = 3ll * device_sm_count();
    const int64_t tokens = 512 * (1 + 2 * items / slots);
    p.slim_tokens = (int)(tokens < 8192 ? tokens : 8192);
}

cudaError_t launch_prefix_finish(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                                 cudaStream_t stream) {
    if (ctas > kMaxRanges) return cudaErrorInvalidValue;
    return dtype == DCP_F16 ? launch_d<__half>(p, ws, tpi, rows, ctas, stream)
                            : launch_d<__nv_bfloat16>(p, ws, tpi, rows, ctas, stream);
}

}  // namespace dcp
