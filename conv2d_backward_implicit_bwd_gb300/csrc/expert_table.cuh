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
    int32_t off[kMaxExperts + 1];   // expert e owns rows [off[e], off[e + 1])
    int32_t tile[kMaxExperts + 1];  // first tile of expert e; tile[experts] = all tiles
    __device__ __forceinline__ int len(int e) const { return off[e + 1] - off[e]; }
};

// Filled by one warp.  `per`: rows per tile, `mult`: tiles per block of `per`
// rows.  Offsets below an earlier one or out of [0, rows] are recorded as a
// fault and read as the running maximum clamped to that range: the experts'
// rows stay disjoint and inside the tensors whatever the offsets hold.
__device__ __forceinline__ void build_expert_table(ExpertTable &t, const int32_t *offsets, int experts, int rows,
                                                   int per, int mult, int32_t *status) {
    const int lane = threadIdx.x & 31;
    int top = 0;  // largest offset so far
    for (int e0 = 0; e0 <= experts; e0 += 32) {
        const int e = e0 + lane;
        const int raw = e <= experts ? offsets[e] : 0;
        int most = max(top, raw);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, most, d);
            if (lane >= d) most = max(most, v);
        }
        top = __shfl_sync(0xffffffffu, most, 31);
        const int o = min(most, rows);
        if (e <= experts) {
            if (o != raw) record_status(status, kDevFaultIndex);
            t.off[e] = o;
        }
    }
    __syncwarp();
    int base = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
        const int e = e0 + lane;
        const int n = e < experts ? (int)(((int64_t)t.len(e) + per - 1) / per) * mult : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (e < experts) t.tile[e] = base + incl - n;
        base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) t.tile[experts] = base;
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

}  // namespace cbd
