// group_table.cuh -- the ragged groups of a grouped linear, as every CTA of its kernels holds
// them in shared memory.  The group offsets live in device memory (the routing of a
// mixture-of-experts layer computes them there, and the host never sees them), so each CTA
// turns them into prefix counts of row tiles itself, with one warp.
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
};

// Inclusive sums over the warp's lanes, of two values at once.
__device__ __forceinline__ void warp_sums(int& a, int& b) {
    const int lane = static_cast<int>(lane_id());
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, a, d), y = __shfl_up_sync(0xFFFFFFFFu, b, d);
        if (lane >= d) {
            a += x;
            b += y;
        }
    }
}

// One chunk of offsets that are out of order or out of range: clamped to the rows and to the
// running maximum.
static __device__ __noinline__ int2 repair_offsets(int cur, int next, int top, int rows, uint32_t* err) {
    const int lane = static_cast<int>(lane_id());
    if (lane == 0) atomicOr(err, kErrGroups);
    cur = max(min(cur, rows), top);
    next = max(min(next, rows), top);
    for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, cur, d);
        if (lane >= d) cur = max(cur, v);
    }
    next = max(next, cur);
    const int right = __shfl_down_sync(0xFFFFFFFFu, cur, 1);
    return make_int2(cur, lane < 31 ? right : next);
}

// One whole warp.  offsets == nullptr: `groups` equal groups (rows a multiple of groups).
// counts[e], where given: the sum of count(m_f) over the groups f before e, counts[groups] that of
// all.  Every kernel of a grouped linear begins with this, with cold instruction caches, so the code is
// kept short: 32 groups a turn, and what repairs bad offsets out of line.
template <typename F>
__device__ __forceinline__ void build_group_table(GroupTable& t, const int32_t* offsets, int groups, int rows, uint32_t* err,
                                                  int32_t* counts, F count) {
    const int lane = static_cast<int>(lane_id());
    const int even = offsets == nullptr ? rows / groups : 0;
    int top = 0, sum = 0, sum2 = 0;   // carried from turn to turn
    auto load = [&](int e) { return offsets != nullptr ? __ldg(offsets + min(e, groups)) : min(e, groups) * even; };
    int ahead = load(lane), ahead_next = load(lane + 1);   // of the turn to come
#pragma unroll 1
    for (int base = 0; base <= groups; base += 32) {
        const int e = base + lane;
        int cur = ahead, next = ahead_next;
        ahead = load(e + 32);
        ahead_next = load(e + 33);
        if (__any_sync(0xFFFFFFFFu, cur < top || cur > rows || next < cur || next > rows)) {
            const int2 good = repair_offsets(cur, next, top, rows, err);
            cur = good.x;
            next = good.y;
        }
        const int m = next - cur;   // zero from the last group on
        int n = (m + 127) >> 7, n2 = e < groups ? count(m) : 0;
        const int own = n, own2 = n2;
        warp_sums(n, n2);
        if (e <= groups) {
            t.start[e] = cur;
            t.tiles[e] = sum + n - own;
            if (counts != nullptr) counts[e] = sum2 + n2 - own2;
        }
        sum += __shfl_sync(0xFFFFFFFFu, n, 31);
        sum2 += __shfl_sync(0xFFFFFFFFu, n2, 31);
        top = __shfl_sync(0xFFFFFFFFu, next, 31);
    }
    __syncwarp();
}

__device__ __forceinline__ void build_group_table(GroupTable& t, const int32_t* offsets, int groups, int rows, uint32_t* err) {
    build_group_table(t, offsets, groups, rows, err, nullptr, [](int) { return 0; });
}

// a / b and a % b of tile counts.  Short code rather than the general division's: a float quotient
// and one correction either way, exact for a < 2^22.
__device__ __forceinline__ int small_div(int a, int b, int* rest) {
    if (a >= 1 << 22) {
        *rest = a % b;
        return a / b;
    }
    int q = static_cast<int>(__fdividef(static_cast<float>(a), static_cast<float>(b)));
    int r = a - q * b;
    if (r < 0) {
        --q;
        r += b;
    }
    if (r >= b) {
        ++q;
        r -= b;
    }
    *rest = r;
    return q;
}

// The group that holds tile, row or cost u: the last e with prefix[e] <= u, for u < prefix[groups].
template <typename T>
__device__ __forceinline__ int find_group(const T* prefix, int groups, T u) {
    int lo = 0, hi = groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace mxfp4
