// ep_groups.cuh -- rows grouped by expert: the table of groups that the expert kernels build in shared memory.
#pragma once

#include "ep_common.cuh"

namespace ep {

// Where the rows of every expert lie (see include/ep.h, expert products).
struct Groups {
    const int32_t* count;  // [groups]
    const int32_t* begin;  // [groups], or NULL: group g begins at g * group_rows
    int64_t num_rows;
    int32_t group_rows;
    int32_t groups;
};

struct Group {
    int32_t begin, count;
};

// Group g, cut to the rows that exist; one that does not fit sets EP_ERR_CAPACITY.
__device__ __forceinline__ Group load_group(const Groups& s, int g, int32_t* status) {
    const int64_t b = s.begin ? s.begin[g] : static_cast<int64_t>(g) * s.group_rows;
    int64_t c = s.count[g];
    const int64_t room = s.begin ? s.num_rows - b : s.group_rows;
    if (c < 0 || (c > 0 && (b < 0 || c > room))) {
        report(status, EP_ERR_CAPACITY);
        c = c < 0 || b < 0 || room < 0 ? 0 : room;
    }
    return {static_cast<int32_t>(c ? b : 0), static_cast<int32_t>(c)};
}

// Exclusive prefix sum of one value per thread over a block of THREADS threads; `sums` has THREADS / 32
// words of shared memory.  Returns this thread's prefix; *total gets the block's sum.  In 64 bits: groups that
// overlap can hold more rows together than there are, and the sum is what shows it.
template <int THREADS>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* sums, int64_t* total) {
    int64_t scan = v;
#pragma unroll
    for (int o = 1; o < kWarpSize; o <<= 1) {
        const int64_t u = __shfl_up_sync(kFullMask, scan, o);
        if (lane_id() >= o) scan += u;
    }
    if (lane_id() == kWarpSize - 1) sums[threadIdx.x / kWarpSize] = scan;
    __syncthreads();
    int64_t base = scan - v, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / kWarpSize; ++w) {
        if (w < static_cast<int>(threadIdx.x / kWarpSize)) base += sums[w];
        all += sums[w];
    }
    *total = all;
    return base;
}

// Last group g with before[g] <= at (before ascending, before[0] = 0).
__device__ __forceinline__ int find_group(const int32_t* before, int groups, int at) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= at) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace ep
