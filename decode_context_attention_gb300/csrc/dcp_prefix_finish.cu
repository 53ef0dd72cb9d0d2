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

// A row's weights are 2^(s - m + kBias): fp16's smallest normal is 2^-14, and a largest
// weight of up to 2^15 keeps those of a long tail (dcp_chunk_attention_tc.cu).
constexpr float kGrow = 8.f;
template <typename T>
constexpr float kBias = std::is_same<T, __half>::value ? 7.f : 0.f;

template <int D>
struct Slim {
    static constexpr int WD = D == 256 ? 2 : 1;       // warps that share a tile's columns
    static constexpr int DW = D / WD;                 // columns of a warp
    static constexpr int kPitch = D * 2 + 64;         // bytes of a staged query row: no bank conflicts
    // of 16 rows: the queries, then the outputs
    static constexpr int kRowBytes = 16 * D * 4;
    static_assert(16 * kPitch <= kRowBytes, "queries lie where the outputs go");
    static constexpr int kSmem = 4 / WD * kRowBytes;
};

// Where the parts of a common item lie: slots of the chunk kernel's partials, or (n = -1) the plan's rows.
struct Parts {
    int n;
    unsigned short slot[kMaxRanges + 1];
};

// The parts of the item, by one warp: the range that holds its first tile by two rounds of 32 at once.
__device__ __noinline__ void find_parts(const ChunkPos* pos, int ctas, const ChunkPos& item, Parts* parts) {
    const int lane = threadIdx.x & 31;
    auto begun = [&](const ChunkPos& x) {
        return x.b != item.b ? x.b < item.b : x.rh != item.rh ? x.rh < item.rh : x.qt != item.qt ? x.qt < item.qt : x.tile == 0;
    };
    const int step = (ctas + 32) / 32;  // of ctas + 1 places; at most 16
    const int n = __popc(__ballot_sync(kAll, lane * step <= ctas && begun(pos[min(lane * step, ctas)])));
    int base = max(n - 1, 0) * step;
    ChunkPos x = pos[min(base + lane, ctas)];
    const int m = __popc(__ballot_sync(kAll, lane < step && base + lane <= ctas && begun(x)));  // c = base + m - 1
    unsigned same = __ballot_sync(kAll, base + lane <= ctas && same_item(x, item));
    if (n == 0 || m == 0 || !(same >> m & 1)) {  // no range begins inside the item
        if (lane == 0) parts->n = -1;
        return;
    }
    if (lane == 0) parts->slot[0] = (unsigned short)(2 * (base + m - 1) + (same >> (m - 1) & 1 ? 0 : 1));
    int count = 1;
    for (int skip = m;; skip = 0) {
        // a range that lies empty inside the item left nothing
        int next_tile = __shfl_down_sync(kAll, x.tile, 1);
        bool next_same = lane < 31 && (same >> (lane + 1) & 1);
        if (lane == 31 && base + 32 <= ctas) {
            const ChunkPos y = pos[base + 32];
            next_tile = y.tile;
            next_same = same_item(y, item);
        }
        const bool in = lane >= skip && base + lane < ctas && (same >> lane & 1);
        const unsigned on = __ballot_sync(kAll, in && !(next_same && next_tile == x.tile));
        if (on >> lane & 1) parts->slot[count + __popc(on & ((1u << lane) - 1u))] =
                (unsigned short)(2 * (base + lane));
        count += __popc(on);
        if (!(same >> 31) || base + 32 >= ctas) break;
        base += 32;
        x = pos[min(base + lane, ctas)];
        same = __ballot_sync(kAll, base + lane <= ctas && same_item(x, item));
    }
    if (lane == 0) parts->n = count;
}

// The joined row so far: base-2 log-sum-exp of the largest part, sum of the weights, and
// this lane's share of the outputs.
template <int NV>
struct Joined {
    float mx, sum;
    float4 acc[NV];
};
template <int NV>
__device__ __forceinline__ void join(Joined<NV>& a, float z, float weight, const float4 (&o)[NV]) {
    // mx becomes finite, infinite or NaN with the parts: as the formula has it
    const float m = fmaxf(a.mx, z), base = m == -INFINITY ? 0.f : m;
    const float old = exp2_fast(a.mx - base), w = exp2_fast(z - base);
    a.mx = m;
    a.sum = fmaf(a.sum, old, w * weight);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        a.acc[v].x = fmaf(w, o[v].x, a.acc[v].x * old);
        a.acc[v].y = fmaf(w, o[v].y, a.acc[v].y * old);
        a.acc[v].z = fmaf(w, o[v].z, a.acc[v].z * old);
        a.acc[v].w = fmaf(w, o[v].w, a.acc[v].w * old);
    }
}

template <typename P>
__device__ __forceinline__ P* shfl_ptr(P* p, int lane) {
    return reinterpret_cast<P*>(__shfl_sync(kAll, (unsigned long long)p, lane));
}
// 1 / x within 1 ulp.
__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What a lane k < kPlaces knows of row k & (count - 1) of the rows that its warp joins: where
// the result goes (NULL: it is none), and how many parts it has.
constexpr int kPlaces = 8;
struct JoinRow {
    unsigned char* out;
    float* lse;
    int parts;
};
// A part's outputs times its weight, the base-2 logarithm of their unit, and its weight: 1 beside a log-sum-exp.
struct Part {
    const float* o;
    float z, weight;
};
// The join of a warp's `count` rows (a power of two up to kPlaces), kPlaces parts in flight:
// kPlaces / count of every row's at a time.  part(n): where the lane's row's n-th part lies,
// in global or shared memory.  (Each lane works out its own row's places, which all lanes
// then read: the instructions of a part that are not its loads come once, not eight times.)
template <typename T, int D, class Get>
__device__ __forceinline__ void join_rows(const PrefixParams& p, int count, const JoinRow& row, Get part) {
    constexpr int NV = (D + 127) / 128;
    const int lane = threadIdx.x & 31;
    const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
    Joined<NV> a[kPlaces];
#pragma unroll
    for (int e = 0; e < kPlaces; ++e) {
        a[e].mx = -INFINITY;
        a[e].sum = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) a[e].acc[v] = none;
    }
    const int step = kPlaces / count, mine = lane / count;
    const int most = (int)__reduce_max_sync(kAll, lane < kPlaces ? (unsigned)row.parts : 0u);
#pragma unroll 1
    for (int i = 0; i < most; i += step) {
        Part x = {nullptr, -INFINITY, 0.f};
        if (lane < kPlaces && i + mine < row.parts) x = part(i + mine);
        float4 o[kPlaces][NV];
#pragma unroll
        for (int e = 0; e < kPlaces; ++e) {
            const float* at = shfl_ptr(x.o, e);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                o[e][v] = at && 4 * lane + 128 * v < D ? *reinterpret_cast<const float4*>(at + 4 * lane + 128 * v) : none;
        }
#pragma unroll
        for (int e = 0; e < kPlaces; ++e)
            join<NV>(a[e], __shfl_sync(kAll, x.z, e), __shfl_sync(kAll, x.weight, e), o[e]);
    }
    if (count <= 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) join<NV>(a[e], a[e + 4].mx, a[e + 4].sum, a[e + 4].acc);
    }
    if (count <= 2) {
#pragma unroll
        for (int e = 0; e < 2; ++e) join<NV>(a[e], a[e + 2].mx, a[e + 2].sum, a[e + 2].acc);
    }
    if (count <= 1) join<NV>(a[0], a[1].mx, a[1].sum, a[1].acc);
    float mx = 0.f, sum = 0.f;
#pragma unroll
    for (int e = 0; e < kPlaces; ++e) {
        unsigned char* out = shfl_ptr(row.out, e);
        if (lane == e) {
            mx = a[e].mx;
            sum = a[e].sum;
        }
        if (e >= count || !out) continue;
        const float inv = a[e].sum == 0.f ? 0.f : reciprocal(a[e].sum);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (4 * lane + 128 * v < D) {
                const float4 x = a[e].acc[v];
                *reinterpret_cast<uint2*>(out + 2 * (4 * lane + 128 * v)) =
                    make_uint2(f32_to_pair(make_float2(x.x * inv, x.y * inv), T()),
                               f32_to_pair(make_float2(x.z * inv, x.w * inv), T()));
            }
    }
    if (lane < count && row.out) {
        const float lse2 = sum == 0.f ? -INFINITY : mx + log2f(sum);
        *row.lse = p.base2 ? lse2 : lse2 * kLn2;
    }
}
__device__ __forceinline__ unsigned char* out_row(const PrefixParams& p, int r, int64_t t, int h) {
    return p.o + (int64_t)r * p.o_sn + t * p.o_st + (int64_t)h * p.o_sh;
}
__device__ __forceinline__ float* out_lse(const PrefixParams& p, int r, int64_t t, int h) {
    return p.lse + (int64_t)r * p.l_sn + t * p.l_st + (int64_t)h * p.l_sh;
}

// ---------------------------------------------------------------------------
// slim own parts
// ---------------------------------------------------------------------------

// Rows of tokens that are not there, of a page outside of the pool or behind the last token.
__device__ const uint4 g_zero_row[64] = {};

__device__ __noinline__ int share_out_of_line(int n, int r, int N) { return rank_share(n, r, N); }

// Item (request, rank, KV head) by 1 << wlog warps of the CTA, its group number `group`.
template <typename T, int D>
__device__ __forceinline__ void slim_part(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas,
                                          int item, int group, int wlog, unsigned char* smem, Parts* parts) {
    using S = Slim<D>;
    constexpr int WD = S::WD, DW = S::DW;
    constexpr int KC = D / 32, VC = DW / 64;  // 16-byte pieces of a key and a value row that a lane takes
    __shared__ float row_m[64], row_l[64];
    __shared__ unsigned poisons[4][4];  // by group: tokens of the masked tiles whose V row is not finite
    const int wpi = 1 << wlog, threads = 32 << wlog;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & (wpi - 1), g = lane >> 2, c = lane & 3;
    const int tid = 32 * warp + lane;  // within the group
    // (a barrier for one warp, too: what tests for it would come twice)
    auto sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(threads) : "memory"); };
    const int b = item / (p.N * p.Hkv), rh = item - b * (p.N * p.Hkv), r = rh / p.Hkv, hkv = rh - r * p.Hkv;
    const Planned q = load_planned(p.slim + 2 * (int64_t)b);
    if (q.n == 0) return;
    bool joined = q.kind == kOwn;
    Planned common;
    common.start = common.n = 0;
    if (joined) common = load_request(p, q.common);
    const int nrows = q.n * p.gq;
    auto seen = [&](int j) { return share_out_of_line(p.causal ? q.L - q.n + j + 1 : q.L, r, p.N); };
    const int lim0 = seen(0), lim_last = q.n == 1 ? lim0 : seen(q.n - 1);
    const int64_t table = table_at(p, q, r, b);
    // row blocks (1 << rlog), and tiles between them
    const int xlog = wlog - (WD - 1), wx_all = 1 << xlog;
    const int rlog = min(nrows <= 16 ? 0 : nrows <= 32 ? 1 : 2, xlog), wt = wx_all >> rlog;
    const int wd = warp >> xlog, wx = warp & (wx_all - 1), blk = wx & ((1 << rlog) - 1), first = wx >> rlog;
    smem += group * (wx_all * S::kRowBytes);
    float* const rm = row_m + group * (16 * wx_all);
    float* const rl = row_l + group * (16 * wx_all);
    unsigned* const poison = poisons[group];
#pragma unroll 1
    for (int id = tid; id < (16 << rlog) * (D / 8); id += threads) {
        const int row = id / (D / 8), u = id % (D / 8);
        const int j = row / p.gq;
        const uint4* at = g_zero_row;
        if (row < nrows)
            at = reinterpret_cast<const uint4*>(p.q + (int64_t)(q.start + j) * p.q_st +
                                                (int64_t)(hkv * p.gq + row - j * p.gq) * p.q_sh);
        *reinterpret_cast<uint4*>(smem + row * S::kPitch + 16 * u) = __ldg(at + u);
    }
    if (tid < 4) poison[tid] = 0u;
    // scores enter with the scale's sign, so that the maximum is that of the scaled ones
    const float sign = p.sm_scale < 0.f ? -1.f : 1.f, qs = fabsf(p.sm_scale) * kLog2e;
    int lim[2] = {lim0, lim0};
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int row = 16 * blk + g + 8 * i;
        int x = lim0;
        if (q.n > 1) x = seen(row / p.gq);
        if (row >= nrows) x = 0;
        if (i) lim[1] = x;
        else lim[0] = x;
    }
    // lane i (and i + 16) knows where the i-th token of a tile lies; a row's pieces are the lanes'
    const unsigned char* const kbase = p.k + (int64_t)r * p.k_sn + (int64_t)hkv * p.k_sh;
    const unsigned char* const vbase = p.v + (int64_t)r * p.v_sn + (int64_t)hkv * p.v_sh;
    const unsigned char *krow, *vrow;
    auto page_at = [&](int t) -> int {
        const int i = t + (lane & 15);
        return i < lim_last ? page_in(p, table, i) : -1;
    };
    auto rows_at = [&](int t, int page) {
        const int slot = (t + (lane & 15)) & ((1 << p.page_shift) - 1);
        const unsigned char* zero = reinterpret_cast<const unsigned char*>(g_zero_row);
        krow = page < 0 ? zero : kbase + (int64_t)page * p.k_sp + (int64_t)slot * p.k_st;
        vrow = page < 0 ? zero : vbase + (int64_t)page * p.v_sp + (int64_t)slot * p.v_st;
    };
    uint4 k[2][KC], v[4][VC];
    auto load_k = [&]() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint4* at = reinterpret_cast<const uint4*>(shfl_ptr(krow, g + 8 * e)) + c;
#pragma unroll
            for (int x = 0; x < KC; ++x) k[e][x] = __ldg(at + 4 * x);
        }
    };
    auto load_v = [&]() {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4* at = reinterpret_cast<const uint4*>(shfl_ptr(vrow, 2 * c + (e & 1) + 8 * (e >> 1))) + DW / 8 * wd + g;
#pragma unroll
            for (int x = 0; x < VC; ++x) v[e][x] = __ldg(at + 8 * x);
        }
    };
    float o[8 * VC][4];
#pragma unroll
    for (int i = 0; i < 8 * VC; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int t = 16 * first;
    rows_at(t, page_at(t));
    load_k();
    sync();
    const unsigned char* qa = smem + (16 * blk + g) * S::kPitch + 16 * c;
#pragma unroll 1
    while (t < lim_last) {
        load_v();
        const int next = t + 16 * wt;
        const int page = page_at(next);
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
        rows_at(next, page);
        load_k();  // (behind the last tile: of the zero row)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[e][x] *= sign;
        const bool masked = t + 16 > lim0;
        if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (t + 8 * e + 2 * c + (x & 1) >= lim[x >> 1]) s[e][x] = -INFINITY;
        }
        float mx[2];
        bool grow[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            grow[i] = (mx[i] - ref[i]) * qs > kGrow || (ref[i] == -INFINITY && mx[i] > -INFINITY);
        }
        // (a row's maximum has grown only if that of one of its lanes' has)
        if (__any_sync(kAll, grow[0] || grow[1])) {
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
        for (int i = 0; i < 2; ++i) {
            const float m = ref[i] == -INFINITY ? 0.f : ref[i];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int x = 2 * i; x < 2 * i + 2; ++x) {
                    // (-infinity times a scale of 0 is no weight)
                    s[e][x] = s[e][x] == -INFINITY ? 0.f : exp2_fast(fmaf(s[e][x] - m, qs, kBias<T>));
                    l[i] += s[e][x];
                }
        }
        if (masked && lim0 < lim_last) {
            // a value that some rows may not see must not reach them as 0 * inf
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                bool bad = false;
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                    const uint4 w = v[e][x];
                    bad |= pair_nonfinite<T>(w.x) || pair_nonfinite<T>(w.y) || pair_nonfinite<T>(w.z) ||
                           pair_nonfinite<T>(w.w);
                }
                if (bad) {
#pragma unroll
                    for (int x = 0; x < VC; ++x) {
                        const uint4 w = v[e][x];
                        v[e][x] = make_uint4(pair_finite<T>(w.x), pair_finite<T>(w.y), pair_finite<T>(w.z),
                                             pair_finite<T>(w.w));
                    }
                    // below 96, as an item's rows are at most 64 tokens' and what they see differs by less
                    const int at = t - (lim0 & ~15) + 2 * c + (e & 1) + 8 * (e >> 1);
                    if (at < 128) atomicOr(&poison[at >> 5], 1u << (at & 31));
                }
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
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(kAll, l[i], 1);
        l[i] += __shfl_xor_sync(kAll, l[i], 2);
    }
    sync();  // every warp is done with the queries
    // the warps' shares of a row: wt of them, 16 << rlog rows apart
    float* os = reinterpret_cast<float*>(smem);  // [wx_all][16][D]
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int at = 16 * wx + g + 8 * i;
        if (wd == 0 && c == 0) {
            rm[at] = ref[i] == -INFINITY ? -INFINITY : fmaf(ref[i], qs, -kBias<T>);
            rl[at] = l[i];
        }
        // lane (g, c) holds columns 64 x + 16 c + [0, 16) of its warp's
#pragma unroll
        for (int x = 0; x < VC; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int j = 4 * (y & 1), z = 2 * i + (y >> 1);
                *reinterpret_cast<float4*>(os + at * D + DW * wd + 64 * x + 16 * c + 4 * y) =
                    make_float4(o[8 * x + j][z], o[8 * x + j + 1][z], o[8 * x + j + 2][z], o[8 * x + j + 3][z]);
            }
    }
    sync();
    if ((poison[0] | poison[1] | poison[2] | poison[3]) != 0u) {
        // what the zeroed values give to the rows that do see them, in the unit of a share that has seen something
#pragma unroll 1
        for (int row = tid; row < nrows; row += threads) {
            const int j = row / p.gq;
            const T* qrow = reinterpret_cast<const T*>(p.q + (int64_t)(q.start + j) * p.q_st +
                                                       (int64_t)(hkv * p.gq + row - j * p.gq) * p.q_sh);
            int at = row;
            while (rm[at] == -INFINITY && at + (16 << rlog) < 16 * wx_all) at += 16 << rlog;
            if (rm[at] != -INFINITY)
                add_nonfinite<T, float>(p, r, table, hkv, qrow, lim0 & ~15, poison, 4, seen(j), rm[at], os + at * D);
        }
        sync();
    }
    // what follows reads what the chunk kernel left
    asm volatile("griddepcontrol.wait;" ::: "memory");
    joined = joined && q.start >= common.start && q.start + q.n <= common.start + common.n;  // (groups out of order)
    int qt0 = 0;
    if (joined) {
        qt0 = (q.start - common.start) / tpi;
        const int last = q.n == 1 ? qt0 : (q.start + q.n - 1 - common.start) / tpi;
#pragma unroll 1
        for (int k = warp; qt0 + k <= last; k += wpi) {  // two at most
            const ChunkPos x = {q.common, rh, qt0 + k, 0};
            find_parts(ws.pos, ctas, x, &parts[2 * group + k]);
        }
        sync();
    }
#pragma unroll 1
    for (int row0 = warp; row0 < nrows; row0 += kPlaces * wpi) {
        const int left = (nrows - row0 + wpi - 1) >> wlog;
        const int count = left > 4 ? 8 : left > 2 ? 4 : left;
        const int row = row0 + wpi * (lane & (count - 1));
        const bool real = row < nrows;
        const int j = real ? row / p.gq : 0, h = hkv * p.gq + (real ? row - j * p.gq : 0), tok = q.start + j;
        const int block = joined ? (tok - common.start) / tpi - qt0 : 0;
        const Parts& from = parts[2 * group + block];
        const bool cut = joined && from.n >= 0;
        const int64_t at = cut ? (int64_t)(tok - common.start - (qt0 + block) * tpi) * p.gq + (h - hkv * p.gq)
                               : ((int64_t)r * p.T + tok) * p.H + h;
        JoinRow x;
        x.out = real ? out_row(p, r, tok, h) : nullptr;
        x.lse = out_lse(p, r, tok, h);
        x.parts = !real ? 0 : wt + (!joined ? 0 : cut ? from.n : 1);
        join_rows<T, D>(p, count, x, [&](int n) -> Part {
            if (n < wt) {
                const int share = row + (n * 16 << rlog);
                return {os + share * D, rm[share], rl[share]};
            }
            const int64_t i = cut ? (int64_t)from.slot[n - wt] * rows + at : at;
            return {(cut ? ws.o : p.wo) + i * D, (cut ? ws.lse : p.wl)[i], 1.f};
        });
    }
}

// ---------------------------------------------------------------------------
// the join of the parts that the chunk kernel has computed
// ---------------------------------------------------------------------------

// Range `c` of the chunk kernel: the items of own parts that begin in it and are joined
// or cut; a CTA takes every `slices`-th of their rows' eights.
template <typename T, int D>
__device__ void join_rest(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int c, int slice,
                          int slices, Parts* parts) {
    constexpr int kWarps = kFinishThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the next kernel of the stream waits for this one only: it must not end before the chunk kernel has
    asm volatile("griddepcontrol.wait;" ::: "memory");
    ChunkPos x = ws.pos[c];
    const ChunkPos end = ws.pos[c + 1];
    if (x.b >= p.requests) return;  // common parts follow the requests' own
    if (x.tile > 0) {               // begun in an earlier range
        if (same_item(x, end)) return;
        x = next_item(p, x, tpi);
    }
#pragma unroll 1
    for (; x.b < p.requests && !(same_item(x, end) && end.tile == 0); x = next_item(p, x, tpi)) {
        const Planned q = load_request(p, x.b);
        const int r = x.rh / p.Hkv, hkv = x.rh % p.Hkv, j0 = x.qt * tpi;
        const int nrows = min(tpi, q.n - j0) * p.gq;
        const bool cut = same_item(x, end);
        bool joined = q.kind == kOwn;
        Planned common;
        if (joined) {
            common = load_request(p, q.common);
            joined = q.start >= common.start && q.start + q.n <= common.start + common.n;  // (groups out of order)
        }
        if (!joined && q.kind == kAlone && !cut) continue;  // written by the chunk kernel itself
        const int qt0 = joined ? (q.start + j0 - common.start) / tpi : 0;
        __syncthreads();  // the item before is done with `parts`
        if (warp == 0) find_parts(ws.pos, ctas, x, &parts[0]);
        else if (joined && warp <= 2) {
            const ChunkPos y = {q.common, x.rh, qt0 + warp - 1, 0};
            find_parts(ws.pos, ctas, y, &parts[warp]);
        }
        __syncthreads();
        const int own_n = parts[0].n < 0 ? 1 : parts[0].n;
#pragma unroll 1
        for (int row0 = (slice * kWarps + warp) * kPlaces; row0 < nrows; row0 += slices * kWarps * kPlaces) {
            const int row = row0 + (lane & (kPlaces - 1));
            const bool real = row < nrows;
            const int j = real ? row / p.gq : 0, h = hkv * p.gq + (real ? row - j * p.gq : 0), tok = q.start + j0 + j;
            const int block = joined ? (tok - common.start) / tpi - qt0 : 0;
            const int64_t whole = ((int64_t)r * p.T + tok) * p.H + h;
            const int64_t within = (int64_t)(tok - common.start - (qt0 + block) * tpi) * p.gq + (h - hkv * p.gq);
            JoinRow g;
            g.out = real ? out_row(p, r, tok, h) : nullptr;
            g.lse = out_lse(p, r, tok, h);
            g.parts = !real ? 0 : own_n + (!joined ? 0 : parts[1 + block].n < 0 ? 1 : parts[1 + block].n);
            join_rows<T, D>(p, kPlaces, g, [&](int n) -> Part {
                const bool own = n < own_n;
                const Parts& from = parts[own ? 0 : 1 + block];
                if (from.n < 0) {  // (own rows lie behind the common ones)
                    const int64_t i = whole + (own ? (int64_t)p.N * p.T * p.H : 0);
                    return {p.wo + i * D, p.wl[i], 1.f};
                }
                const int64_t i = (int64_t)from.slot[own ? n : n - own_n] * rows + (own ? row : within);
                return {ws.o + i * D, ws.lse[i], 1.f};
            });
        }
        if (cut) break;  // the range ends inside it
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kFinishThreads, D == 64 ? 4 : D == 128 ? 3 : 2)
    prefix_finish_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ ChunkPartials ws, int tpi, int rows, int ctas, int blocks, int wlog,
                         int slices) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Parts parts[8];
    if ((int)blockIdx.x < blocks) {
        const int group = (int)(threadIdx.x >> 5) >> wlog;
        const int item = (int)blockIdx.x * (4 >> wlog) + group;
        if (item < p.requests * p.N * p.Hkv) slim_part<T, D>(p, ws, tpi, rows, ctas, item, group, wlog, smem, parts);
    } else {
        const int k = blockIdx.x - blocks;
        join_rest<T, D>(p, ws, tpi, rows, ctas, k / slices, k % slices, slices, parts);
    }
}

template <typename T, int D>
cudaError_t launch(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, cudaStream_t stream) {
    const auto kernel = prefix_finish_kernel<T, D>;
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv;
    const int wpi = p.slim_warps;
    const int64_t blocks = (items + 4 / wpi - 1) / (4 / wpi);
    const int slices = 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks + ctas * slices));
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
    return cudaLaunchKernelEx(&cfg, kernel, p, ws, tpi, rows, ctas, (int)blocks, wpi == 4 ? 2 : wpi - 1, slices);
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

// Warps of an item: alone, a warp streams longest for the set-up it pays; with fewer items
// than warps fit at once they share its tiles.  Items of more than 16 rows want a warp for
// each 16.  An own part is slim up to the rows of its warps, and up to as many tokens of a
// rank as keep them from outlasting the others: with fewer items, a long part is better
// cut over the SMs.
void slim_limits(PrefixParams& p) {
    const int64_t items = (int64_t)p.requests * p.N * p.Hkv, sms = device_sm_count();
    const int64_t drafts = ((int64_t)p.T + p.requests - 1) / p.requests;  // new tokens of a request, about
    int warps = items >= 6 * sms ? 1 : items >= 3 * sms ? 2 : 4;
    if (drafts * p.gq > 16) warps = 4;
    if (p.D == 256 && warps < 2) warps = 2;  // a row's columns are two warps'
    p.slim_warps = warps;
    p.slim_rows = 16 * warps / (p.D == 256 ? 2 : 1);
    const int64_t tokens = 512 * (1 + 2 * items / (3 * sms));
    p.slim_tokens = (int)(tokens < 8192 ? tokens : 8192);
}

cudaError_t launch_prefix_finish(const PrefixParams& p, const ChunkPartials& ws, int tpi, int rows, int ctas, int dtype,
                                 cudaStream_t stream) {
    if (ctas > kMaxRanges) return cudaErrorInvalidValue;
    return dtype == DCP_F16 ? launch_d<__half>(p, ws, tpi, rows, ctas, stream)
                            : launch_d<__nv_bfloat16>(p, ws, tpi, rows, ctas, stream);
}

}  // namespace dcp
