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
    int32_t tile[kMaxExperts + 1];  // first tile of the i-th expert in tile order; tile[experts] = all tiles
    uint16_t order[kMaxExperts];    // experts by falling cost of their tiles
    __device__ __forceinline__ int len(int e) const { return off[e + 1] - off[e]; }
};

// Rows in equal chunks of at most `per`, rounded up to 32.
__device__ __forceinline__ int chunk_rows(int len, int per) {
    const int chunks = (len + per - 1) / per;
    return ((len + chunks - 1) / chunks + 31) & ~31;
}

enum ExpertTiles : int {
    kTilesByRows,   // ceil(rows / per) x mult tiles, dearer ones (more rows each) first
    kTilesByDepth,  // mult tiles each, more rows first
    kTilesNonEmpty, // as kTilesByDepth without the experts that have no rows
    kTilesInOrder,  // ceil(rows / per) x mult tiles in the order of the experts (`order` is not written)
};

// Step 1, all threads of the block: the offsets as they are.
__device__ __forceinline__ void load_expert_offsets(ExpertTable &t, const int32_t *offsets, int experts) {
    for (int e = threadIdx.x; e <= experts; e += blockDim.x) t.off[e] = offsets[e];
}

// Step 2, one warp, after a block barrier.  Offsets below an earlier one or out of [0, rows] are
// recorded as a fault and read as the running maximum clamped to that range:
// the experts' rows stay disjoint and inside the tensors whatever the offsets
// hold.  Tiles go by falling cost in eight classes, so that the last ones to be
// handed out are the short ones.
__device__ __forceinline__ void build_expert_table(ExpertTable &t, int experts, int rows, int per, int mult,
                                                   ExpertTiles kind, int32_t *status) {
    constexpr int CLASSES = 8;
    const int lane = threadIdx.x & 31;
    int top = 0, longest = 0;  // largest offset so far
    for (int e0 = 0; e0 <= experts; e0 += 32) {
        const int e = e0 + lane;
        const int raw = e <= experts ? t.off[e] : 0;
        int most = max(top, raw);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, most, d);
            if (lane >= d) most = max(most, v);
        }
        const int o = min(most, rows);
        int before = __shfl_up_sync(0xffffffffu, o, 1);
        if (lane == 0) before = min(top, rows);
        if (e > 0 && e <= experts) longest = max(longest, o - before);
        top = __shfl_sync(0xffffffffu, most, 31);
        if (e <= experts) {
            if (o != raw) record_status(status, kDevFaultIndex);
            t.off[e] = o;
        }
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    __syncwarp();
    auto cls = [&](int e) {
        const int len = t.len(e);
        const int cost = kind == kTilesByRows ? (len ? chunk_rows(len, per) : 0) : len;
        const int most = kind == kTilesByRows ? per : longest;
        return CLASSES - 1 - min(CLASSES - 1, (int)(((int64_t)max(cost - 1, 0) * CLASSES) / max(most, 1)));
    };
    int base[CLASSES];
#pragma unroll
    for (int c = 0; c < CLASSES; ++c) base[c] = 0;
    const int sorted = kind == kTilesInOrder ? 0 : experts;
    for (int e0 = 0; e0 < sorted; e0 += 32) {
        const int mine = e0 + lane < experts ? cls(e0 + lane) : -1;
#pragma unroll
        for (int c = 0; c < CLASSES; ++c) base[c] += __popc(__ballot_sync(0xffffffffu, mine == c));
    }
    int sum = 0;
#pragma unroll
    for (int c = 0; c < CLASSES; ++c) {
        const int n = base[c];
        base[c] = sum;
        sum += n;
    }
    for (int e0 = 0; e0 < sorted; e0 += 32) {
        const int mine = e0 + lane < experts ? cls(e0 + lane) : -1;
#pragma unroll
        for (int c = 0; c < CLASSES; ++c) {
            const uint32_t m = __ballot_sync(0xffffffffu, mine == c);
            if (mine == c) t.order[base[c] + __popc(m & ((1u << lane) - 1))] = (uint16_t)(e0 + lane);
            base[c] += __popc(m);
        }
    }
    __syncwarp();
    int tiles = 0;
    for (int i0 = 0; i0 < experts; i0 += 32) {
        const int i = i0 + lane;
        int n = 0;
        if (i < experts) {
            const int len = t.len(kind == kTilesInOrder ? i : t.order[i]);
            n = kind == kTilesByRows || kind == kTilesInOrder ? (int)(((int64_t)len + per - 1) / per) * mult : kind == kTilesNonEmpty && len == 0 ? 0 : mult;
        }
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += v;
        }
        if (i < experts) t.tile[i] = tiles + incl - n;
        tiles += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) t.tile[experts] = tiles;
}

// Position in tile order of the expert that tile t belongs to: the last i with
// tile[i] <= t (experts without tiles share a bound with the next one).
__device__ __forceinline__ int position_of_tile(const ExpertTable &tab, int experts, int t) {
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
