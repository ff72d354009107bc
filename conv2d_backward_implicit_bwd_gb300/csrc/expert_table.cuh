// expert_table.cuh -- the tile table of a launch grouped by expert, built by
// each block from the device-side offsets: the host never learns the rows of
// an expert, so a router's output feeds the products without a copy back.
#pragma once
#include <stdint.h>

#include "device_util.cuh"
#include "internal.h"
#include "train.h"

namespace cbd {

struct ExpertTable {
    int32_t begin[kMaxExperts];      // first row of the expert
    int32_t len[kMaxExperts];        // its rows
    int32_t tile[kMaxExperts + 1];   // first tile of the expert; tile[experts] = all tiles
};

// Filled by one warp.  `per`: rows per tile, `mult`: tiles per block of `per`
// rows.  An expert whose offsets are out of [0, rows] or fall below an earlier
// offset is empty and recorded as a fault, so that the experts' rows are
// disjoint and no later access leaves the tensors.
__device__ __forceinline__ void build_expert_table(ExpertTable &t, const int32_t *offsets, int experts, int rows,
                                                   int per, int mult, int32_t *status) {
    const int lane = threadIdx.x & 31;
    int base_tile = 0, top = 0;  // top: largest offset so far
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        int lo = e < experts ? offsets[e] : 0, hi = e < experts ? offsets[e + 1] : 0;
        int most = max(top, lo);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, most, d);
            if (lane >= d) most = max(most, v);
        }
        top = __shfl_sync(0xffffffffu, most, 31);
        if (e < experts && (lo < most || hi < lo || hi > rows)) {
            record_status(status, kDevFaultIndex);
            lo = hi = 0;
        }
        int n = (int)(((int64_t)(hi - lo) + per - 1) / per) * mult;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (e < experts) {
            t.begin[e] = lo;
            t.len[e] = hi - lo;
            t.tile[e] = base_tile + incl - n;
        }
        base_tile += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) t.tile[experts] = base_tile;
}

// Expert of tile t (tile[e] <= t < tile[e + 1]), by bisection.
__device__ __forceinline__ int expert_of_tile(const ExpertTable &tab, int experts, int t) {
    int lo = 0, hi = experts - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.tile[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// Rows of no expert: [0, fill_lo) and [fill_hi, rows).
__device__ __forceinline__ void fill_bounds(const int32_t *offsets, int experts, int rows, int &fill_lo, int &fill_hi) {
    fill_lo = min(max(offsets[0], 0), rows);
    fill_hi = min(max(offsets[experts], fill_lo), rows);
}

}  // namespace cbd
