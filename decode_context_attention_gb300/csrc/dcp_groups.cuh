// dcp_groups.cuh -- groups of requests whose first tokens are common, and the
// round-robin share of a rank in pages.
#pragma once

#include "dcp_device.cuh"

namespace dcp {

// Consecutive requests [group_start[g], group_start[g + 1]) share their first
// prefix_lens[g] tokens.  Only whole pages are shared, and only where every rank
// has them: floor(prefix / (N * page_size)) table entries on each rank.
struct Groups {
    int G;
    const int* start;     // [G + 1], non-decreasing
    const int* prefix;    // [G]
    int N, page_shift;
    int max_seq_len, max_entries;
};

// The groups' arrays in shared memory, when there is room for them: a lookup is a search of
// dependent loads.  All threads of the CTA; ends with a barrier.
constexpr int kGroupsHeld = 1024;
struct GroupsHeld {
    int start[kGroupsHeld + 1], prefix[kGroupsHeld];
};
__device__ __forceinline__ Groups hold_groups(const Groups& x, GroupsHeld* held) {
    Groups y = x;
    if (x.G > 0 && x.G <= kGroupsHeld) {
        for (int g = threadIdx.x; g <= x.G; g += blockDim.x) {
            held->start[g] = x.start[g];
            if (g < x.G) held->prefix[g] = x.prefix[g];
        }
        y.start = held->start;
        y.prefix = held->prefix;
    }
    __syncthreads();
    return y;
}

// Table entries on every rank that the requests of group g have in common.
__device__ __forceinline__ int common_entries(const Groups& x, int g) {
    const int p = min(max(x.prefix[g], 0), x.max_seq_len);
    return min((p / x.N) >> x.page_shift, x.max_entries);
}

// The group of request b, or -1: the last one that starts at or before b, when it
// ends behind b.  Whatever `start` holds, a group returned starts in [0, b].
__device__ __forceinline__ int group_of(const Groups& x, int b) {
    int lo = 0, hi = x.G;  // groups before lo start at or before b
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (x.start[mid] <= b) lo = mid + 1;
        else hi = mid;
    }
    if (lo == 0 || x.start[lo - 1] < 0 || x.start[lo] <= b) return -1;
    return lo - 1;
}

// The request whose pages b has for its first `entries` table entries: b itself,
// with none, outside of groups and for a group's first request.
struct Member {
    int first, entries;
};
__device__ __forceinline__ Member member_of(const Groups& x, int b) {
    const int g = group_of(x, b);
    if (g < 0) return {b, 0};
    const int first = x.start[g];
    return {first, first == b ? 0 : common_entries(x, g)};
}

}  // namespace dcp
