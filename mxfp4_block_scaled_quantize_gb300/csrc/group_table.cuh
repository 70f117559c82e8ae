// group_table.cuh -- the ragged groups of a grouped linear, as every CTA of its kernels holds
// them in shared memory.  The group offsets live in device memory (the routing of a
// mixture-of-experts layer computes them there, and the host never sees them), so each CTA
// turns them into prefix counts of row tiles itself: one warp, a few hundred cycles.
//
// Offsets come from outside and are not trusted: each is clamped to [0, rows] and to its
// predecessor, which keeps every index derived from the table inside the buffers, and a
// table that needed clamping is recorded in the device error word.
#pragma once

#include <cstdint>

#include "launch.h"
#include "ptx.cuh"

namespace mxfp4 {

struct GroupTable {
    int32_t start[kMaxGroups + 1];    // first row of each group, and the last group's end
    int32_t tiles[kMaxGroups + 1];    // 128-row tiles of the groups before, and of all
    int32_t tiles2[kMaxGroups + 1];   // the same for 256-row tiles
};

// One whole warp.  offsets == nullptr: `groups` equal groups (rows a multiple of groups).
__device__ __forceinline__ void build_group_table(GroupTable& t, const int32_t* offsets, int groups, int rows,
                                                  uint32_t* err) {
    const int lane = static_cast<int>(lane_id());
    const int per = (groups + 1 + 31) >> 5;
    const int first = lane * per, last = min(first + per, groups + 1);
    const int even = rows / groups;
    // starts: clamp, then the running maximum
    int top = 0;
    bool bad = false;
    for (int e = first; e < last; ++e) {
        const int o = offsets != nullptr ? __ldg(offsets + e) : e * even;
        top = max(top, min(max(o, 0), rows));
        bad = bad || o != top;
        t.start[e] = top;
    }
    int carry = top;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, carry, d);
        if (lane >= d) carry = max(carry, v);
    }
    carry = __shfl_up_sync(0xFFFFFFFFu, carry, 1);
    if (lane == 0) carry = 0;
    for (int e = first; e < last && t.start[e] < carry; ++e) {
        t.start[e] = carry;
        bad = true;
    }
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(err, kErrGroups);
    __syncwarp();
    // tiles: exclusive prefix sums
    int n = 0, n2 = 0;
    for (int e = first; e < min(last, groups); ++e) {
        const int m = t.start[e + 1] - t.start[e];
        n += (m + 127) >> 7;
        n2 += (m + 255) >> 8;
    }
    int sum = n, sum2 = n2;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d), v2 = __shfl_up_sync(0xFFFFFFFFu, sum2, d);
        if (lane >= d) {
            sum += v;
            sum2 += v2;
        }
    }
    sum -= n;
    sum2 -= n2;
    for (int e = first; e < last; ++e) {
        t.tiles[e] = sum;
        t.tiles2[e] = sum2;
        if (e < groups) {
            const int m = t.start[e + 1] - t.start[e];
            sum += (m + 127) >> 7;
            sum2 += (m + 255) >> 8;
        }
    }
    __syncwarp();
}

// The group that holds tile (or row) u: the last e with prefix[e] <= u, for u < prefix[groups].
__device__ __forceinline__ int find_group(const int32_t* prefix, int groups, int u) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace mxfp4
