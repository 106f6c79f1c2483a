// scan.cuh -- sums over the sequences of a call, in one block of threads.
#pragma once

#include <stdint.h>

namespace pkv {

constexpr unsigned kAllLanes = 0xffffffffu;
constexpr unsigned kFull30 = 1u << 30; // sums saturate here: past every capacity

__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, kFull30); }

// Exclusive prefix sums of (a, b) over the block's threads, and their totals.
__device__ __forceinline__ void block_scan(unsigned &a, unsigned &b, unsigned &ta, unsigned &tb,
                                           uint2 *warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    unsigned x = a, y = b;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned u = __shfl_up_sync(kAllLanes, x, d), v = __shfl_up_sync(kAllLanes, y, d);
        if (lane >= d) {
            x = add_sat(x, u);
            y = add_sat(y, v);
        }
    }
    unsigned ex = __shfl_up_sync(kAllLanes, x, 1), ey = __shfl_up_sync(kAllLanes, y, 1);
    if (lane == 0) ex = ey = 0;
    if (lane == 31) warp_sums[warp] = make_uint2(x, y);
    __syncthreads();
    // every warp sums the warps before it, and all of them
    uint2 w = lane < warps ? warp_sums[lane] : make_uint2(0, 0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const unsigned u = __shfl_up_sync(kAllLanes, w.x, d), v = __shfl_up_sync(kAllLanes, w.y, d);
        if (lane >= d) {
            w.x = add_sat(w.x, u);
            w.y = add_sat(w.y, v);
        }
    }
    const unsigned bx = __shfl_sync(kAllLanes, w.x, warp > 0 ? warp - 1 : 0);
    const unsigned by = __shfl_sync(kAllLanes, w.y, warp > 0 ? warp - 1 : 0);
    ta = __shfl_sync(kAllLanes, w.x, 31);
    tb = __shfl_sync(kAllLanes, w.y, 31);
    a = add_sat(ex, warp > 0 ? bx : 0);
    b = add_sat(ey, warp > 0 ? by : 0);
    __syncthreads();
}

// The last s of [0, n) whose start[s] <= x (start is non-decreasing, start[0] <= x).
__device__ __forceinline__ int last_at_or_before(const int *start, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace pkv
