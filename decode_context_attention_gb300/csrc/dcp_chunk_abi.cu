// dcp_chunk_abi.cu -- the extern "C" entry points of the chunk-serving kernels
// declared in include/dcp.h: argument validation on the host and dispatch.
// Nothing here touches device memory: a rejected call launches nothing.
#include <math.h>

#include "dcp.h"
#include "dcp_internal.h"
#include "dcp_validate.h"

using namespace dcp;

namespace {

// A pool of pages [N][num_pages, page_size, Hkv, D] of 2-byte elements.
struct Pool {
    const void* p;
    int64_t sn, sp, st, sh;
    View view(int N, int num_pages, int page_size, int Hkv, int D) const {
        return View(p, (int64_t)D * 2).dim(N, sn * 2).dim(num_pages, sp * 2).dim(page_size, st * 2).dim(Hkv, sh * 2);
    }
};

bool finite(float x) { return x == x && x != INFINITY && x != -INFINITY; }

// The sizes every chunk entry point shares; DCP_OK, or the recorded failure.
dcp_status_t check_batch(const char* who, int dtype, int N, int B, int T, int Hkv, int num_pages, int page_size,
                         int max_pages, int max_seq_len) {
    if (dtype != DCP_F16 && dtype != DCP_BF16)
        return fail(DCP_ERR_UNSUPPORTED_DTYPE, "%s: dtype %d (f16 or bf16 only)", who, dtype);
    if (N < 1 || N > kMaxRanks || B < 0 || T < 0 || Hkv < 1 || max_seq_len < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: sizes N=%d B=%d T=%d Hkv=%d max_seq_len=%d", who, N, B, T, Hkv,
                    max_seq_len);
    if (page_size < 1 || page_size > (1 << 16) || (page_size & (page_size - 1)))
        return fail(DCP_ERR_INVALID_ARG, "%s: page_size %d (a power of two up to 65536)", who, page_size);
    if (num_pages < 1) return fail(DCP_ERR_INVALID_ARG, "%s: num_pages %d", who, num_pages);
    const int64_t lcap = ((int64_t)max_seq_len + N - 1) / N;
    const int64_t need = (lcap + page_size - 1) / page_size;
    if (max_pages < need)
        return fail(DCP_ERR_INVALID_ARG, "%s: page table rows of %d entries; %lld needed for %lld local tokens", who,
                    max_pages, (long long)need, (long long)lcap);
    // (request, rank) pairs and token indices are 32-bit in the kernels
    if ((int64_t)N * B * Hkv >= (1ll << 31) || max_seq_len > (1 << 30) || B >= (1 << 30))
        return fail(DCP_ERR_INVALID_ARG, "%s: N*B*Hkv below 2^31 and max_seq_len up to 2^30 only", who);
    return DCP_OK;
}

int page_shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

dcp_status_t check_heads(const char* who, int T, int H, int Hkv, int D) {
    if (H < 1) return fail(DCP_ERR_INVALID_ARG, "%s: H=%d", who, H);
    if (H % Hkv) return fail(DCP_ERR_HEADS_NOT_DIVISIBLE, "%s: H=%d is not a multiple of Hkv=%d", who, H, Hkv);
    if (H / Hkv > 64) return fail(DCP_ERR_INVALID_ARG, "%s: H/Hkv=%d (up to 64 query heads per KV head)", who, H / Hkv);
    if (D != 64 && D != 128 && D != 256) return fail(DCP_ERR_INVALID_ARG, "%s: D=%d (64, 128 or 256)", who, D);
    // row indices are 32-bit in the kernels, up to a tile past the last row
    if ((int64_t)T * H >= (1ll << 30)) return fail(DCP_ERR_INVALID_ARG, "%s: too many rows (T * H >= 2^30)", who);
    return DCP_OK;
}

void fill_batch(ChunkParams& p, int N, int B, int T, int H, int Hkv, int D, int max_seq_len, int page_size,
                int num_pages, const int* bt, int64_t bt_sn, int64_t bt_sb, const int* query_start,
                const int* seq_lens, const Pool& k, const Pool& v) {
    p = ChunkParams{};
    p.N = N; p.B = B; p.T = T; p.H = H; p.Hkv = Hkv; p.D = D; p.gq = H / Hkv;
    p.max_seq_len = max_seq_len;
    p.page_shift = page_shift_of(page_size); p.num_pages = num_pages;
    p.causal = 1;
    p.query_start = query_start; p.seq_lens = seq_lens;
    p.bt = bt; p.bt_sn = bt_sn; p.bt_sb = bt_sb;
    p.k = (unsigned char*)k.p; p.k_sn = k.sn * 2; p.k_sp = k.sp * 2; p.k_st = k.st * 2; p.k_sh = k.sh * 2;
    p.v = (unsigned char*)v.p; p.v_sn = v.sn * 2; p.v_sp = v.sp * 2; p.v_st = v.st * 2; p.v_sh = v.sh * 2;
}

bool any_overlap(const View& out, std::initializer_list<const View*> others) {
    for (const View* v : others)
        if (overlap(out, *v)) return true;
    return false;
}

// Whether the K and V rows of two pools are disjoint: pools apart from each
// other, or interleaved in one buffer (the same strides, rows side by side).
bool pools_disjoint(const Pool& k, const Pool& v, const View& kp, const View& vp) {
    if (!kp.rows_disjoint() || !vp.rows_disjoint()) return false;
    if (!overlap(kp, vp)) return true;
    for (int i = 0; i < kp.nd; ++i)
        if (kp.size[i] > 1 && kp.stride[i] != vp.stride[i]) return false;
    const bool k_first = (uintptr_t)k.p < (uintptr_t)v.p;
    View both(k_first ? k.p : v.p, kp.inner);
    for (int i = 0; i < kp.nd; ++i) both.dim(kp.size[i], kp.stride[i]);
    return both.dim(2, (int64_t)(k_first ? vp.base - kp.base : kp.base - vp.base)).rows_disjoint();
}

// dcp_extend_attention_paged and dcp_prefix_attention_paged (G groups; 0: none).
dcp_status_t attend(const char* who, int dtype, int N, int B, int T, int H, int Hkv, int D, const void* q, int64_t q_st,
                    int64_t q_sh, const Pool& pk, const Pool& pv, int num_pages, int page_size, const int* block_table,
                    int64_t bt_sn, int64_t bt_sb, int max_pages, const int* query_start, const int* seq_lens,
                    int max_seq_len, int G, const int* group_start, const int* prefix_lens, float sm_scale, int causal,
                    void* o, int64_t o_sn, int64_t o_st, int64_t o_sh, float* lse, int64_t l_sn, int64_t l_st,
                    int64_t l_sh, int lse_base, void* workspace, size_t workspace_bytes, void* stream) {
    if (const dcp_status_t s = check_batch(who, dtype, N, B, T, Hkv, num_pages, page_size, max_pages, max_seq_len))
        return s;
    if (const dcp_status_t s = check_heads(who, T, H, Hkv, D)) return s;
    if (!finite(sm_scale)) return fail(DCP_ERR_INVALID_ARG, "%s: sm_scale is not finite", who);
    if (lse_base != DCP_LSE_BASE_E && lse_base != DCP_LSE_BASE_2)
        return fail(DCP_ERR_INVALID_ARG, "%s: lse_base %d", who, lse_base);
    // the plan's (request, rank, head) triples are counted in 32 bits, too
    if (G < 0 || (G && (int64_t)N * ((int64_t)G + B) * Hkv >= (1ll << 30)))
        return fail(DCP_ERR_INVALID_ARG, "%s: G=%d (N * (G + B) * Hkv below 2^30)", who, G);
    if (B == 0 || T == 0) return ok();
    if (!q || !pk.p || !pv.p || !block_table || !query_start || !seq_lens || !o || !lse ||
        (G && (!group_start || !prefix_lens)))
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({q_st, q_sh, pk.sn, pk.sp, pk.st, pk.sh, pv.sn, pv.sp, pv.st, pv.sh, bt_sn, bt_sb, o_sn, o_st, o_sh, l_sn,
                    l_st, l_sh}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const int64_t rb = (int64_t)D * 2;
    View vq = View(q, rb).dim(T, q_st * 2).dim(H, q_sh * 2);
    View kp = pk.view(N, num_pages, page_size, Hkv, D), vp = pv.view(N, num_pages, page_size, Hkv, D);
    View vo = View(o, rb).dim(N, o_sn * 2).dim(T, o_st * 2).dim(H, o_sh * 2);
    View vl = View(lse, 4).dim(N, l_sn * 4).dim(T, l_st * 4).dim(H, l_sh * 4);
    View qs = View(query_start, 4).dim((int64_t)B + 1, 4), sl = View(seq_lens, 4).dim(B, 4);
    View gs = View(group_start, G ? 4 : 0).dim((int64_t)G + 1, 4), pl = View(prefix_lens, G ? 4 : 0).dim(G, 4);
    View bt = View(block_table, 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4).dim(max_pages, 4);
    if (!all_fit({&vq, &kp, &vp, &vo, &vl, &bt}))
        return fail(DCP_ERR_INVALID_ARG, "%s: an operand's strides span more than 2^56 bytes", who);
    if (vq.align() < 16 || kp.align() < 16 || vp.align() < 16 || vo.align() < 16)
        return fail(DCP_ERR_MISALIGNED, "%s: q, o and page rows must start on 16-byte boundaries", who);
    if ((uintptr_t)lse % 4 || (uintptr_t)block_table % 4 || (uintptr_t)query_start % 4 || (uintptr_t)seq_lens % 4 ||
        (G && ((uintptr_t)group_start % 4 || (uintptr_t)prefix_lens % 4)))
        return fail(DCP_ERR_MISALIGNED, "%s: pointer not aligned to its element type", who);
    for (const View* out : {&vo, &vl})
        if (any_overlap(*out, {&vq, &kp, &vp, &qs, &sl, &bt, &gs, &pl}))
            return fail(DCP_ERR_ALIAS, "%s: an output overlaps an input", who);
    if (overlap(vo, vl) || !vo.rows_disjoint() || !vl.rows_disjoint())
        return fail(DCP_ERR_ALIAS, "%s: outputs overlap", who);
    const size_t need = prefix_attention_workspace(N, B, T, H, Hkv, D, max_seq_len, G);
    if (!workspace || workspace_bytes < need)
        return fail(DCP_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed (%zu given)", who, need,
                    workspace ? workspace_bytes : (size_t)0);
    if ((uintptr_t)workspace % 16) return fail(DCP_ERR_MISALIGNED, "%s: workspace not 16-byte aligned", who);
    if (any_overlap(View(workspace, (int64_t)need), {&vq, &kp, &vp, &vo, &vl, &qs, &sl, &bt, &gs, &pl}))
        return fail(DCP_ERR_ALIAS, "%s: workspace overlaps an operand", who);
    PrefixParams p{};
    fill_batch(p, N, B, T, H, Hkv, D, max_seq_len, page_size, num_pages, block_table, bt_sn, bt_sb, query_start,
               seq_lens, pk, pv);
    p.causal = causal != 0;
    p.base2 = lse_base == DCP_LSE_BASE_2;
    p.sm_scale = sm_scale;
    p.q = (const unsigned char*)q; p.q_st = q_st * 2; p.q_sh = q_sh * 2;
    p.o = (unsigned char*)o; p.o_sn = o_sn * 2; p.o_st = o_st * 2; p.o_sh = o_sh * 2;
    p.lse = lse; p.l_sn = l_sn; p.l_st = l_st; p.l_sh = l_sh;
    p.ws = (unsigned char*)workspace;
    p.requests = B; p.groups = G; p.group_start = group_start; p.prefix_lens = prefix_lens; p.max_pages = max_pages;
    return launched(launch_prefix_attention(p, dtype, (cudaStream_t)stream), who);
}

}  // namespace

extern "C" {

dcp_status_t dcp_qk_norm_rope_append(int dtype, int N, int B, int T, int H, int Hkv, int D,
                                     const void* q, int64_t q_st, int64_t q_sh,
                                     const void* k, int64_t k_st, int64_t k_sh,
                                     const void* v, int64_t v_st, int64_t v_sh,
                                     const void* q_weight, const void* k_weight, float eps,
                                     const float* cos_sin, int num_positions, int rot_dim, int interleaved,
                                     const int* positions,
                                     void* q_out, int64_t qo_st, int64_t qo_sh,
                                     void* k_pages, int64_t kp_sn, int64_t kp_sp, int64_t kp_st, int64_t kp_sh,
                                     void* v_pages, int64_t vp_sn, int64_t vp_sp, int64_t vp_st, int64_t vp_sh,
                                     int num_pages, int page_size,
                                     const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                                     const int* query_start, const int* seq_lens, int max_seq_len, void* stream) {
    const char* who = "dcp_qk_norm_rope_append";
    if (const dcp_status_t s = check_batch(who, dtype, N, B, T, Hkv, num_pages, page_size, max_pages, max_seq_len))
        return s;
    if (H < 1) return fail(DCP_ERR_INVALID_ARG, "%s: H=%d", who, H);
    if (D < 16 || D > 512 || D % 16)
        return fail(DCP_ERR_INVALID_ARG, "%s: D=%d (a multiple of 16 up to 512)", who, D);
    if (rot_dim < 0 || rot_dim > D || rot_dim % 16)
        return fail(DCP_ERR_INVALID_ARG, "%s: rot_dim=%d (a multiple of 16 up to D=%d)", who, rot_dim, D);
    if (rot_dim && num_positions < 1) return fail(DCP_ERR_INVALID_ARG, "%s: num_positions=%d", who, num_positions);
    if (!finite(eps) || eps < 0.f) return fail(DCP_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", who);
    if ((int64_t)T * ((int64_t)H + 2 * (int64_t)Hkv) >= (1ll << 31))
        return fail(DCP_ERR_INVALID_ARG, "%s: too many head rows (T * (H + 2 Hkv) >= 2^31)", who);
    if (B == 0 || T == 0) return ok();
    if (!q || !k || !v || !q_out || !k_pages || !v_pages || !block_table || !query_start || !seq_lens ||
        (rot_dim && (!cos_sin || !positions)))
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({q_st, q_sh, k_st, k_sh, v_st, v_sh, qo_st, qo_sh, kp_sn, kp_sp, kp_st, kp_sh, vp_sn, vp_sp, vp_st,
                    vp_sh, bt_sn, bt_sb}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const int64_t rb = (int64_t)D * 2;
    const Pool pk{k_pages, kp_sn, kp_sp, kp_st, kp_sh}, pv{v_pages, vp_sn, vp_sp, vp_st, vp_sh};
    View vq = View(q, rb).dim(T, q_st * 2).dim(H, q_sh * 2);
    View vk = View(k, rb).dim(T, k_st * 2).dim(Hkv, k_sh * 2);
    View vv = View(v, rb).dim(T, v_st * 2).dim(Hkv, v_sh * 2);
    View vo = View(q_out, rb).dim(T, qo_st * 2).dim(H, qo_sh * 2);
    View kp = pk.view(N, num_pages, page_size, Hkv, D), vp = pv.view(N, num_pages, page_size, Hkv, D);
    View qw = View(q_weight, q_weight ? rb : 0), kw = View(k_weight, k_weight ? rb : 0);
    View cs = View(cos_sin, (int64_t)rot_dim * 4).dim(num_positions, (int64_t)rot_dim * 4);
    View ps = View(positions, rot_dim ? 4 : 0).dim(T, 4);
    View qs = View(query_start, 4).dim((int64_t)B + 1, 4), sl = View(seq_lens, 4).dim(B, 4);
    View bt = View(block_table, 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4).dim(max_pages, 4);
    if (!all_fit({&vq, &vk, &vv, &vo, &kp, &vp, &bt}))
        return fail(DCP_ERR_INVALID_ARG, "%s: an operand's strides span more than 2^56 bytes", who);
    if (vq.align() < 16 || vk.align() < 16 || vv.align() < 16 || vo.align() < 16 || kp.align() < 16 || vp.align() < 16)
        return fail(DCP_ERR_MISALIGNED, "%s: head rows must start on 16-byte boundaries", who);
    if ((uintptr_t)q_weight % 16 || (uintptr_t)k_weight % 16 || (rot_dim && (uintptr_t)cos_sin % 16))
        return fail(DCP_ERR_MISALIGNED, "%s: norm weights and cos_sin must be 16-byte aligned", who);
    if ((rot_dim && (uintptr_t)positions % 4) || (uintptr_t)block_table % 4 || (uintptr_t)query_start % 4 ||
        (uintptr_t)seq_lens % 4)
        return fail(DCP_ERR_MISALIGNED, "%s: pointer not aligned to its element type", who);
    const bool inplace = q_out == q && (T <= 1 || qo_st == q_st) && (H <= 1 || qo_sh == q_sh);
    if (!inplace && overlap(vo, vq))
        return fail(DCP_ERR_ALIAS, "%s: q_out overlaps q other than as q itself", who);
    // in place, q may be the head slice of a fused projection that k and v are
    // slices of too: its extent covers them, but rows side by side stay apart
    auto side_by_side = [&](const View& other) {
        if (other.size[0] > 1 && other.stride[0] != vo.stride[0]) return false;
        uintptr_t alo, ahi, blo, bhi;
        View a = vo, b = other;
        a.size[0] = b.size[0] = 1;
        a.extent(alo, ahi);
        b.extent(blo, bhi);
        const int64_t token = T > 1 ? vo.stride[0] : kMaxSpan;
        return (ahi <= blo && (int64_t)(bhi - alo) <= token) || (bhi <= alo && (int64_t)(ahi - blo) <= token);
    };
    for (const View* in : {&vk, &vv})
        if (overlap(vo, *in) && !side_by_side(*in)) return fail(DCP_ERR_ALIAS, "%s: q_out overlaps k or v", who);
    if (any_overlap(vo, {&qw, &kw, &cs, &ps, &qs, &sl, &bt, &kp, &vp}))
        return fail(DCP_ERR_ALIAS, "%s: q_out overlaps an input or the pages", who);
    for (const View* out : {&kp, &vp})
        if (any_overlap(*out, {&vq, &vk, &vv, &qw, &kw, &cs, &ps, &qs, &sl, &bt}))
            return fail(DCP_ERR_ALIAS, "%s: the pages overlap an input", who);
    if (!vo.rows_disjoint() || !pools_disjoint(pk, pv, kp, vp))
        return fail(DCP_ERR_ALIAS, "%s: rows of an output overlap one another", who);
    AppendParams a{};
    fill_batch(a.c, N, B, T, H, Hkv, D, max_seq_len, page_size, num_pages, block_table, bt_sn, bt_sb, query_start,
               seq_lens, pk, pv);
    a.c.q = (const unsigned char*)q; a.c.q_st = q_st * 2; a.c.q_sh = q_sh * 2;
    a.rot = rot_dim; a.interleaved = interleaved != 0; a.num_positions = num_positions; a.eps = eps;
    a.kn = (const unsigned char*)k; a.kn_st = k_st * 2; a.kn_sh = k_sh * 2;
    a.vn = (const unsigned char*)v; a.vn_st = v_st * 2; a.vn_sh = v_sh * 2;
    a.qo = (unsigned char*)q_out; a.qo_st = qo_st * 2; a.qo_sh = qo_sh * 2;
    a.qw = (const unsigned char*)q_weight; a.kw = (const unsigned char*)k_weight;
    a.cos_sin = cos_sin; a.positions = positions;
    return launched(launch_append(a, dtype, (cudaStream_t)stream), who);
}

size_t dcp_extend_attention_workspace_size(int N, int B, int T, int H, int Hkv, int D, int max_seq_len) {
    if (N < 1 || N > kMaxRanks || B < 0 || T < 0 || H < 1 || Hkv < 1 || H % Hkv || H / Hkv > 64 || max_seq_len < 0 ||
        (D != 64 && D != 128 && D != 256))
        return 0;
    return chunk_attention_workspace(N, B, T, H, Hkv, D, max_seq_len);
}

dcp_status_t dcp_extend_attention_paged(int dtype, int N, int B, int T, int H, int Hkv, int D,
                                        const void* q, int64_t q_st, int64_t q_sh,
                                        const void* k_pages, int64_t k_sn, int64_t k_sp, int64_t k_st, int64_t k_sh,
                                        const void* v_pages, int64_t v_sn, int64_t v_sp, int64_t v_st, int64_t v_sh,
                                        int num_pages, int page_size,
                                        const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                                        const int* query_start, const int* seq_lens, int max_seq_len,
                                        float sm_scale, int causal,
                                        void* o, int64_t o_sn, int64_t o_st, int64_t o_sh,
                                        float* lse, int64_t l_sn, int64_t l_st, int64_t l_sh,
                                        int lse_base, void* workspace, size_t workspace_bytes, void* stream) {
    return attend("dcp_extend_attention_paged", dtype, N, B, T, H, Hkv, D, q, q_st, q_sh,
                  Pool{k_pages, k_sn, k_sp, k_st, k_sh}, Pool{v_pages, v_sn, v_sp, v_st, v_sh}, num_pages, page_size,
                  block_table, bt_sn, bt_sb, max_pages, query_start, seq_lens, max_seq_len, 0, nullptr, nullptr,
                  sm_scale, causal, o, o_sn, o_st, o_sh, lse, l_sn, l_st, l_sh, lse_base, workspace, workspace_bytes,
                  stream);
}

size_t dcp_prefix_attention_workspace_size(int N, int B, int T, int H, int Hkv, int D, int max_seq_len, int G) {
    if (G < 0 || dcp_extend_attention_workspace_size(N, B, T, H, Hkv, D, max_seq_len) == 0) return 0;
    return prefix_attention_workspace(N, B, T, H, Hkv, D, max_seq_len, G);
}

dcp_status_t dcp_prefix_attention_paged(int dtype, int N, int B, int T, int H, int Hkv, int D,
                                        const void* q, int64_t q_st, int64_t q_sh,
                                        const void* k_pages, int64_t k_sn, int64_t k_sp, int64_t k_st, int64_t k_sh,
                                        const void* v_pages, int64_t v_sn, int64_t v_sp, int64_t v_st, int64_t v_sh,
                                        int num_pages, int page_size,
                                        const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                                        const int* query_start, const int* seq_lens, int max_seq_len,
                                        int G, const int* group_start, const int* prefix_lens,
                                        float sm_scale, int causal,
                                        void* o, int64_t o_sn, int64_t o_st, int64_t o_sh,
                                        float* lse, int64_t l_sn, int64_t l_st, int64_t l_sh,
                                        int lse_base, void* workspace, size_t workspace_bytes, void* stream) {
    return attend("dcp_prefix_attention_paged", dtype, N, B, T, H, Hkv, D, q, q_st, q_sh,
                  Pool{k_pages, k_sn, k_sp, k_st, k_sh}, Pool{v_pages, v_sn, v_sp, v_st, v_sh}, num_pages, page_size,
                  block_table, bt_sn, bt_sb, max_pages, query_start, seq_lens, max_seq_len, G, group_start, prefix_lens,
                  sm_scale, causal, o, o_sn, o_st, o_sh, lse, l_sn, l_st, l_sh, lse_base, workspace, workspace_bytes,
                  stream);
}

dcp_status_t dcp_attention_weights_paged(int dtype, int N, int B, int T, int H, int Hkv, int D,
                                         const void* q, int64_t q_st, int64_t q_sh,
                                         const void* k_pages, int64_t k_sn, int64_t k_sp, int64_t k_st, int64_t k_sh,
                                         int num_pages, int page_size,
                                         const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                                         const int* query_start, const int* seq_lens, int max_seq_len,
                                         float sm_scale,
                                         const float* lse, int64_t l_st, int64_t l_sh, int lse_base,
                                         float* acc, int64_t a_sn, int64_t a_sb, int64_t a_sh, void* stream) {
    const char* who = "dcp_attention_weights_paged";
    if (const dcp_status_t s = check_batch(who, dtype, N, B, T, Hkv, num_pages, page_size, max_pages, max_seq_len))
        return s;
    if (const dcp_status_t s = check_heads(who, T, H, Hkv, D)) return s;
    if (!finite(sm_scale)) return fail(DCP_ERR_INVALID_ARG, "%s: sm_scale is not finite", who);
    if (lse_base != DCP_LSE_BASE_E && lse_base != DCP_LSE_BASE_2)
        return fail(DCP_ERR_INVALID_ARG, "%s: lse_base %d", who, lse_base);
    const int64_t cap = ((int64_t)max_seq_len + N - 1) / N;
    if (((cap + 63) / 64) * N * B * Hkv >= (1ll << 31))
        return fail(DCP_ERR_INVALID_ARG, "%s: too many token tiles (2^31 or more)", who);
    if (B == 0 || T == 0 || cap == 0) return ok();
    if (!q || !k_pages || !block_table || !query_start || !seq_lens || !lse || !acc)
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({q_st, q_sh, k_sn, k_sp, k_st, k_sh, bt_sn, bt_sb, l_st, l_sh, a_sn, a_sb, a_sh}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const Pool pk{k_pages, k_sn, k_sp, k_st, k_sh}, none{nullptr, 0, 0, 0, 0};
    View vq = View(q, (int64_t)D * 2).dim(T, q_st * 2).dim(H, q_sh * 2);
    View kp = pk.view(N, num_pages, page_size, Hkv, D);
    View vl = View(lse, 4).dim(T, l_st * 4).dim(H, l_sh * 4);
    View va = View(acc, cap * 4).dim(N, a_sn * 4).dim(B, a_sb * 4).dim(Hkv, a_sh * 4);
    View qs = View(query_start, 4).dim((int64_t)B + 1, 4), sl = View(seq_lens, 4).dim(B, 4);
    View bt = View(block_table, 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4).dim(max_pages, 4);
    if (!all_fit({&vq, &kp, &vl, &va, &bt}))
        return fail(DCP_ERR_INVALID_ARG, "%s: an operand's strides span more than 2^56 bytes", who);
    if (vq.align() < 16 || kp.align() < 16)
        return fail(DCP_ERR_MISALIGNED, "%s: q and page rows must start on 16-byte boundaries", who);
    if ((uintptr_t)lse % 4 || (uintptr_t)acc % 4 || (uintptr_t)block_table % 4 || (uintptr_t)query_start % 4 ||
        (uintptr_t)seq_lens % 4)
        return fail(DCP_ERR_MISALIGNED, "%s: pointer not aligned to its element type", who);
    if (any_overlap(va, {&vq, &kp, &vl, &qs, &sl, &bt}))
        return fail(DCP_ERR_ALIAS, "%s: acc overlaps an input", who);
    if (!va.rows_disjoint()) return fail(DCP_ERR_ALIAS, "%s: acc rows overlap one another", who);
    ChunkParams p;
    fill_batch(p, N, B, T, H, Hkv, D, max_seq_len, page_size, num_pages, block_table, bt_sn, bt_sb, query_start,
               seq_lens, pk, none);
    p.base2 = lse_base == DCP_LSE_BASE_2;
    p.sm_scale = sm_scale;
    p.q = (const unsigned char*)q; p.q_st = q_st * 2; p.q_sh = q_sh * 2;
    p.lse = const_cast<float*>(lse); p.l_st = l_st; p.l_sh = l_sh;
    p.acc = acc; p.a_sn = a_sn; p.a_sb = a_sb; p.a_sh = a_sh;
    return launched(launch_chunk_weights(p, dtype, (cudaStream_t)stream), who);
}

dcp_status_t dcp_cache_evict_paged(int dtype, int N, int B, int Hkv, int D,
                                   void* k_pages, int64_t k_sn, int64_t k_sp, int64_t k_st, int64_t k_sh,
                                   void* v_pages, int64_t v_sn, int64_t v_sp, int64_t v_st, int64_t v_sh,
                                   int num_pages, int page_size,
                                   const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                                   const int* seq_lens, int max_seq_len,
                                   const float* acc, int64_t a_sn, int64_t a_sb, int64_t a_sh,
                                   const int* keep_lens, int max_keep, int recent,
                                   const int* dst_table, int64_t dt_sn, int64_t dt_sb, int dst_max_pages,
                                   int* kept, int64_t kp_sn, int64_t kp_sb, int64_t kp_sh,
                                   float* acc_out, int64_t ao_sn, int64_t ao_sb, int64_t ao_sh, void* stream) {
    const char* who = "dcp_cache_evict_paged";
    if (const dcp_status_t s = check_batch(who, dtype, N, B, 0, Hkv, num_pages, page_size, max_pages, max_seq_len))
        return s;
    if (D < 8 || D > 1024 || D % 8) return fail(DCP_ERR_INVALID_ARG, "%s: D=%d (a multiple of 8 up to 1024)", who, D);
    if (max_keep < 0 || recent < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: max_keep=%d recent=%d", who, max_keep, recent);
    const int64_t cap = ((int64_t)max_seq_len + N - 1) / N;
    // a request never keeps more than it holds
    if (max_keep > max_seq_len) max_keep = max_seq_len;
    const int64_t kcap = ((int64_t)max_keep + N - 1) / N;
    const int64_t need = (kcap + page_size - 1) / page_size;
    if (dst_max_pages < need)
        return fail(DCP_ERR_INVALID_ARG, "%s: destination table rows of %d entries; %lld needed for %lld local tokens",
                    who, dst_max_pages, (long long)need, (long long)kcap);
    const int64_t rb = (int64_t)D * 2;
    // 8 CTAs a problem, and a few rows a CTA, stay below 2^31 CTAs
    if (8 * (int64_t)N * B * Hkv >= (1ll << 31) || (kcap / 8 + 1) * N * B * Hkv >= (1ll << 31))
        return fail(DCP_ERR_INVALID_ARG, "%s: too many rows to move", who);
    if (B == 0 || cap == 0 || kcap == 0) return ok();
    if (!k_pages || !v_pages || !block_table || !seq_lens || !acc || !keep_lens || !dst_table || !kept || !acc_out)
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({k_sn, k_sp, k_st, k_sh, v_sn, v_sp, v_st, v_sh, bt_sn, bt_sb, a_sn, a_sb, a_sh, dt_sn, dt_sb,
                    kp_sn, kp_sb, kp_sh, ao_sn, ao_sb, ao_sh}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const Pool pk{k_pages, k_sn, k_sp, k_st, k_sh}, pv{v_pages, v_sn, v_sp, v_st, v_sh};
    View kp = pk.view(N, num_pages, page_size, Hkv, D), vp = pv.view(N, num_pages, page_size, Hkv, D);
    View va = View(acc, cap * 4).dim(N, a_sn * 4).dim(B, a_sb * 4).dim(Hkv, a_sh * 4);
    View vk = View(kept, kcap * 4).dim(N, kp_sn * 4).dim(B, kp_sb * 4).dim(Hkv, kp_sh * 4);
    View vu = View(acc_out, kcap * 4).dim(N, ao_sn * 4).dim(B, ao_sb * 4).dim(Hkv, ao_sh * 4);
    View sl = View(seq_lens, 4).dim(B, 4), kl = View(keep_lens, 4).dim(B, 4);
    View bt = View(block_table, 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4).dim(max_pages, 4);
    View dt = View(dst_table, 4).dim(N, dt_sn * 4).dim(B, dt_sb * 4).dim(dst_max_pages, 4);
    if (!all_fit({&kp, &vp, &va, &vk, &vu, &bt, &dt}))
        return fail(DCP_ERR_INVALID_ARG, "%s: an operand's strides span more than 2^56 bytes", who);
    if (kp.align() < 16 || vp.align() < 16)
        return fail(DCP_ERR_MISALIGNED, "%s: page rows must start on 16-byte boundaries", who);
    if ((uintptr_t)acc % 4 || (uintptr_t)kept % 4 || (uintptr_t)acc_out % 4 || (uintptr_t)seq_lens % 4 ||
        (uintptr_t)keep_lens % 4 || (uintptr_t)block_table % 4 || (uintptr_t)dst_table % 4)
        return fail(DCP_ERR_MISALIGNED, "%s: pointer not aligned to its element type", who);
    for (const View* out : {&kp, &vp, &vk, &vu})
        if (any_overlap(*out, {&va, &sl, &kl, &bt, &dt}))
            return fail(DCP_ERR_ALIAS, "%s: an output overlaps an input", who);
    if (overlap(vk, vu) || any_overlap(vk, {&kp, &vp}) || any_overlap(vu, {&kp, &vp}) || !vk.rows_disjoint() ||
        !vu.rows_disjoint())
        return fail(DCP_ERR_ALIAS, "%s: outputs overlap", who);
    if (!pools_disjoint(pk, pv, kp, vp)) return fail(DCP_ERR_ALIAS, "%s: page rows overlap one another", who);
    EvictParams e{};
    fill_batch(e.c, N, B, 0, Hkv, Hkv, D, max_seq_len, page_size, num_pages, block_table, bt_sn, bt_sb, nullptr,
               seq_lens, pk, pv);
    e.c.acc = const_cast<float*>(acc); e.c.a_sn = a_sn; e.c.a_sb = a_sb; e.c.a_sh = a_sh;
    e.row_bytes = (int)rb;
    e.max_keep = max_keep; e.recent = recent; e.keep_lens = keep_lens;
    e.dt = dst_table; e.dt_sn = dt_sn; e.dt_sb = dt_sb;
    e.kept = kept; e.kp_sn = kp_sn; e.kp_sb = kp_sb; e.kp_sh = kp_sh;
    e.acc_out = acc_out; e.ao_sn = ao_sn; e.ao_sb = ao_sb; e.ao_sh = ao_sh;
    return launched(launch_evict(e, (cudaStream_t)stream), who);
}

}  // extern "C"
