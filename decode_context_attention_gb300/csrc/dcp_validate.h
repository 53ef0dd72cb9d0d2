// dcp_validate.h -- host-side argument checks shared by the C entry points:
// element sizes, stride and span limits, strided views with overlap and
// alignment tests, and the error record of this host thread.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>
#include <utility>

#include "dcp.h"

namespace dcp {

// Record a failure (dcp_last_error_message() of this host thread) and return
// its status; clear the record and return DCP_OK; the result of a launch.
dcp_status_t fail(dcp_status_t s, const char* fmt, ...);
dcp_status_t ok();
dcp_status_t launched(cudaError_t e, const char* what);

constexpr int kMaxRanks = 4096;

inline int elem_size(int dtype) {
    switch (dtype) {
        case DCP_F32: return 4;
        case DCP_F16:
        case DCP_BF16: return 2;
        case DCP_FP8_E4M3: return 1;
        default: return 0;
    }
}

// Limits that keep every byte offset in 64 bits: a stride of at most 2^52
// elements (times at most 4 bytes), a payload row of at most 2^30 bytes (row
// and vector offsets are 32-bit in the kernels), and at most 2^56 bytes
// between the first and the last byte an operand's rows can touch.
constexpr int64_t kMaxStride = int64_t(1) << 52;
constexpr int64_t kMaxRowBytes = int64_t(1) << 30;
constexpr int64_t kMaxSpan = int64_t(1) << 56;

// A strided set of rows: `nd` outer dimensions (size, stride in BYTES) and
// `inner` contiguous bytes per row.
struct View {
    uintptr_t base = 0;
    int nd = 0;
    int64_t size[5] = {0, 0, 0, 0, 0};
    int64_t stride[5] = {0, 0, 0, 0, 0};
    int64_t inner = 0;

    View(const void* p, int64_t inner_bytes) : base((uintptr_t)p), inner(inner_bytes) {}
    View& dim(int64_t n, int64_t stride_bytes) {
        size[nd] = n;
        stride[nd] = stride_bytes;
        ++nd;
        return *this;
    }
    bool empty() const {
        for (int i = 0; i < nd; ++i)
            if (size[i] == 0) return true;
        return inner == 0;
    }
    // False when the rows would span more than kMaxSpan bytes (or the span
    // overflows): no device holds that much memory, so such strides are a
    // caller's mistake, and refusing them keeps every address computation
    // below (host and device, 64-bit) free of overflow.
    bool fits() const {
        int64_t s = inner;
        for (int i = 0; i < nd; ++i) {
            if (size[i] <= 1) continue;
            int64_t t;
            if (__builtin_mul_overflow(size[i] - 1, stride[i], &t) || __builtin_add_overflow(s, t, &s))
                return false;
        }
        return s <= kMaxSpan;
    }
    // Byte range [lo, hi) that the rows can touch.
    void extent(uintptr_t& lo, uintptr_t& hi) const {
        lo = base;
        hi = base + (uintptr_t)inner;
        for (int i = 0; i < nd; ++i)
            if (size[i] > 1) hi += (uintptr_t)((size[i] - 1) * stride[i]);
    }
    // True when distinct index tuples address disjoint byte ranges: sorted by
    // stride, every stride spans at least the block of the smaller dimensions.
    bool rows_disjoint() const { return rows_disjoint_with_inner(inner); }
    bool rows_disjoint_with_inner(int64_t row_bytes) const {
        int idx[5];
        int m = 0;
        for (int i = 0; i < nd; ++i)
            if (size[i] > 1) idx[m++] = i;
        for (int a = 1; a < m; ++a)
            for (int b = a; b > 0 && stride[idx[b]] < stride[idx[b - 1]]; --b) std::swap(idx[b], idx[b - 1]);
        int64_t span = row_bytes;
        for (int a = 0; a < m; ++a) {
            const int i = idx[a];
            if (stride[i] < span) return false;
            span = stride[i] * (size[i] - 1) + span;
        }
        return true;
    }
    // Largest power of two (<= 16) dividing every row start.
    int align() const {
        uint64_t bits = (uint64_t)base | 16u;
        for (int i = 0; i < nd; ++i)
            if (size[i] > 1) bits |= (uint64_t)stride[i];
        return (int)(bits & (~bits + 1));
    }
};

inline bool overlap(const View& a, const View& b) {
    if (a.empty() || b.empty()) return false;
    uintptr_t alo, ahi, blo, bhi;
    a.extent(alo, ahi);
    b.extent(blo, bhi);
    return alo < bhi && blo < ahi;
}

// A stride below 0 or above kMaxStride elements.
inline bool bad_stride(std::initializer_list<int64_t> s) {
    for (int64_t v : s)
        if (v < 0 || v > kMaxStride) return true;
    return false;
}

inline bool all_fit(std::initializer_list<const View*> views) {
    for (const View* v : views)
        if (!v->fits()) return false;
    return true;
}

// Widest vector (16, 4 or 2 bytes) that divides the row length and every row
// start of the views given by their alignments.
inline int pick_vb(int row_bytes, int align_a, int align_b, int e) {
    const int a = align_a < align_b ? align_a : align_b;
    if (a % 16 == 0 && row_bytes % 16 == 0) return 16;
    if (a % 4 == 0 && row_bytes % 4 == 0) return 4;
    return e == 2 ? 2 : 4;
}

// fp8 rows are moved in 4- or 16-byte vectors only: the row length and every
// row start must be multiples of 4 bytes (one e4m3 element is one byte).
inline bool fp8_rows_ok(int e, int D, int align_a, int align_b) {
    return e != 1 || (D % 4 == 0 && align_a >= 4 && align_b >= 4);
}

inline int lanes_per_row(int vectors) {
    int l = 1;
    while (l < vectors && l < 32) l <<= 1;
    return l;
}

}  // namespace dcp
