// dcp_pages_abi.cu -- the extern "C" entry points of the page bookkeeping declared
// in include/dcp.h: argument validation on the host and dispatch.  Nothing here
// touches device memory: a rejected call launches nothing.
#include "dcp.h"
#include "dcp_internal.h"
#include "dcp_validate.h"

using namespace dcp;

namespace {

struct Named {
    const char* name;
    View view;
    bool counts = false;  // free_count and free_count_out, which may be one array
};

// What both entry points share: sizes, and the table against them.
dcp_status_t check_sizes(const char* who, int N, int B, int page_size, int num_pages, int max_seq_len, int G,
                         int max_pages, int free_capacity) {
    if (N < 1 || N > kMaxRanks || B < 0 || max_seq_len < 0 || max_seq_len > (1 << 30) || G < 0)
        return fail(DCP_ERR_INVALID_ARG, "%s: sizes N=%d B=%d max_seq_len=%d G=%d", who, N, B, max_seq_len, G);
    if (page_size < 1 || page_size > (1 << 16) || (page_size & (page_size - 1)))
        return fail(DCP_ERR_INVALID_ARG, "%s: page_size %d (a power of two up to 65536)", who, page_size);
    if (num_pages < 1 || free_capacity < 1)
        return fail(DCP_ERR_INVALID_ARG, "%s: num_pages=%d free_capacity=%d", who, num_pages, free_capacity);
    const int64_t lcap = ((int64_t)max_seq_len + N - 1) / N, need = (lcap + page_size - 1) / page_size;
    if (max_pages < need)
        return fail(DCP_ERR_INVALID_ARG, "%s: page table rows of %d entries; %lld needed for %lld local tokens", who,
                    max_pages, (long long)need, (long long)lcap);
    if ((int64_t)N * B >= (1ll << 31) || B >= (1 << 30))
        return fail(DCP_ERR_INVALID_ARG, "%s: N*B below 2^31 only", who);
    return DCP_OK;
}

dcp_status_t check_operands(const char* who, std::initializer_list<Named> in, std::initializer_list<Named> out) {
    for (const auto* l : {&in, &out})
        for (const Named& x : *l) {
            if (!x.view.fits())
                return fail(DCP_ERR_INVALID_ARG, "%s: %s's strides span more than 2^56 bytes", who, x.name);
            if (!x.view.empty() && x.view.align() < (x.view.inner == 8 ? 8 : 4))
                return fail(DCP_ERR_MISALIGNED, "%s: %s not aligned to its element type", who, x.name);
        }
    for (const Named* a = out.begin(); a != out.end(); ++a) {
        if (!a->view.rows_disjoint()) return fail(DCP_ERR_ALIAS, "%s: rows of %s overlap one another", who, a->name);
        for (const Named* b = a + 1; b != out.end(); ++b)
            if (overlap(a->view, b->view)) return fail(DCP_ERR_ALIAS, "%s: %s and %s overlap", who, a->name, b->name);
        for (const Named& b : in) {
            // a rank's count is read and written by the same block
            if (a->counts && b.counts && a->view.base == b.view.base) continue;
            if (overlap(a->view, b.view)) return fail(DCP_ERR_ALIAS, "%s: %s overlaps %s", who, a->name, b.name);
        }
    }
    return DCP_OK;
}

int shift_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

View row4(const void* p, int64_t n) { return View(p, p ? 4 : 0).dim(n, 4); }

}  // namespace

extern "C" {

dcp_status_t dcp_page_reserve(int N, int B, int T, int page_size, int num_pages, int max_seq_len,
                              const int* cached_lens, const int* new_lens,
                              int G, const int* group_start, const int* prefix_lens,
                              int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                              const int* free_pages, int64_t fp_sn, int free_capacity, const int* free_count,
                              int* free_count_out, int* missing, int* query_start, int* seq_lens,
                              int* positions, int64_t* slots, int* requests, void* stream) {
    const char* who = "dcp_page_reserve";
    if (const dcp_status_t s = check_sizes(who, N, B, page_size, num_pages, max_seq_len, G, max_pages, free_capacity))
        return s;
    if (T < 0 || T > (1 << 30)) return fail(DCP_ERR_INVALID_ARG, "%s: T=%d (0 to 2^30)", who, T);
    if (B == 0) return ok();
    if (!cached_lens || !new_lens || !block_table || !free_pages || !free_count || !free_count_out || !missing ||
        !query_start || !seq_lens || (G && (!group_start || !prefix_lens)))
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({bt_sn, bt_sb, fp_sn}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const int64_t g = G;
    if (const dcp_status_t s = check_operands(
            who,
            {{"cached_lens", row4(cached_lens, B)}, {"new_lens", row4(new_lens, B)},
             {"group_start", row4(G ? group_start : nullptr, g + 1)}, {"prefix_lens", row4(G ? prefix_lens : nullptr, g)},
             {"free_pages", View(free_pages, (int64_t)free_capacity * 4).dim(N, fp_sn * 4)},
             {"free_count", row4(free_count, N), true}},
            {{"block_table", View(block_table, (int64_t)max_pages * 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4)},
             {"free_count_out", row4(free_count_out, N), true}, {"missing", row4(missing, N)},
             {"query_start", row4(query_start, (int64_t)B + 1)}, {"seq_lens", row4(seq_lens, B)},
             {"positions", row4(positions, T)}, {"slots", View(slots, slots ? 8 : 0).dim(T, 8)},
             {"requests", row4(requests, T)}}))
        return s;
    PageParams p{};
    p.N = N; p.B = B; p.T = T; p.page_shift = shift_of(page_size); p.num_pages = num_pages; p.max_seq_len = max_seq_len;
    p.G = G; p.group_start = group_start; p.prefix_lens = prefix_lens;
    p.bt = block_table; p.bt_sn = bt_sn; p.bt_sb = bt_sb; p.max_pages = max_pages;
    p.free_pages = const_cast<int*>(free_pages); p.fp_sn = fp_sn; p.free_capacity = free_capacity;
    p.free_count = free_count; p.free_out = free_count_out;
    p.cached_lens = cached_lens; p.new_lens = new_lens; p.missing = missing;
    p.query_start = query_start; p.seq_lens = seq_lens;
    p.positions = positions; p.slots = slots; p.requests = requests;
    return launched(launch_page_reserve(p, (cudaStream_t)stream), who);
}

dcp_status_t dcp_page_release(int N, int B, int page_size, int num_pages, int max_seq_len,
                              const int* seq_lens, const int* keep_lens,
                              int G, const int* group_start, const int* prefix_lens,
                              const int* block_table, int64_t bt_sn, int64_t bt_sb, int max_pages,
                              int* free_pages, int64_t fp_sn, int free_capacity, const int* free_count,
                              int* free_count_out, int* lens_out, void* stream) {
    const char* who = "dcp_page_release";
    if (const dcp_status_t s = check_sizes(who, N, B, page_size, num_pages, max_seq_len, G, max_pages, free_capacity))
        return s;
    if (B == 0) return ok();
    if (!seq_lens || !keep_lens || !block_table || !free_pages || !free_count || !free_count_out ||
        (G && (!group_start || !prefix_lens)))
        return fail(DCP_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (bad_stride({bt_sn, bt_sb, fp_sn}))
        return fail(DCP_ERR_INVALID_ARG, "%s: negative stride or one above 2^52 elements", who);
    const int64_t g = G;
    if (const dcp_status_t s = check_operands(
            who,
            {{"seq_lens", row4(seq_lens, B)}, {"keep_lens", row4(keep_lens, B)},
             {"group_start", row4(G ? group_start : nullptr, g + 1)}, {"prefix_lens", row4(G ? prefix_lens : nullptr, g)},
             {"block_table", View(block_table, (int64_t)max_pages * 4).dim(N, bt_sn * 4).dim(B, bt_sb * 4)},
             {"free_count", row4(free_count, N), true}},
            {{"free_pages", View(free_pages, (int64_t)free_capacity * 4).dim(N, fp_sn * 4)},
             {"free_count_out", row4(free_count_out, N), true}, {"lens_out", row4(lens_out, B)}}))
        return s;
    PageParams p{};
    p.N = N; p.B = B; p.page_shift = shift_of(page_size); p.num_pages = num_pages; p.max_seq_len = max_seq_len;
    p.G = G; p.group_start = group_start; p.prefix_lens = prefix_lens;
    p.bt = const_cast<int*>(block_table); p.bt_sn = bt_sn; p.bt_sb = bt_sb; p.max_pages = max_pages;
    p.free_pages = free_pages; p.fp_sn = fp_sn; p.free_capacity = free_capacity;
    p.free_count = free_count; p.free_out = free_count_out;
    p.lens = seq_lens; p.keep_lens = keep_lens; p.lens_out = lens_out;
    return launched(launch_page_release(p, (cudaStream_t)stream), who);
}

}  // extern "C"
