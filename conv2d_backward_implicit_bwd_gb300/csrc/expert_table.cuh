// expert_table.cuh -- the tile table of a launch grouped by expert, built by
// each block from the device-side offsets (the host never learns the rows of an
// expert, so a router's output feeds the products without a copy back), and the
// ring through which one warp hands decoded tiles to the others.
//
// The start of a launch runs cold: an instruction line costs a fetch from L2, so
// straight code is slow there (a table that sorted the experts by cost in some
// 600 instructions took 6.4 us, this one 0.8 us, at 13 experts).
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

// By one warp: expert e has ceil(rows / per) x mult tiles, with `each` mult tiles
// if it has no rows.  Offsets below an earlier one or out of [0, rows] are recorded as
// a fault and read as the running maximum clamped to that range: the experts'
// rows stay disjoint and inside the tensors whatever the offsets hold.
__device__ __forceinline__ void build_expert_table(ExpertTable &t, const int32_t *offsets, int experts, int rows,
                                                   uint32_t per, int mult, bool each, int32_t *status) {
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int e = lane; e <= experts; e += 32) t.off[e] = offsets[e];
    __syncwarp();
    int top = 0, tiles = 0;  // last offset, tiles so far
#pragma unroll 1
    for (int e0 = 0; e0 <= experts; e0 += 32) {
        const int e = e0 + lane;
        int o = e <= experts ? t.off[e] : rows;
        int before = __shfl_up_sync(0xffffffffu, o, 1);
        if (lane == 0) before = top;
        if (__any_sync(0xffffffffu, o < before || o > rows)) {
            const int raw = o;
            o = max(o, top);
#pragma unroll 1
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, o, d);
                if (lane >= d) o = max(o, v);
            }
            o = min(o, rows);
            if (e <= experts && o != raw) record_status(status, kDevFaultIndex);
            before = __shfl_up_sync(0xffffffffu, o, 1);
            if (lane == 0) before = top;
        }
        top = __shfl_sync(0xffffffffu, o, 31);
        // tiles of expert e - 1
        const uint32_t len = e > 0 && e <= experts ? (uint32_t)(o - before) : 0u;
        int n = (int)((len + per - 1) / per) * mult;
        if (each && len == 0 && e > 0 && e <= experts) n = mult;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, n, d);
            if (lane >= d) n += v;
        }
        if (e <= experts) {
            t.off[e] = o;
            t.tile[e] = tiles + n;
        }
        tiles += __shfl_sync(0xffffffffu, n, 31);
    }
    __syncwarp();
}

// The same after pdl_wait().  What comes before it overlaps the kernel before this
// one, so an empty list goes through the code first and its instructions are there
// when the offsets are (``zero``: any 0 in shared memory).
__device__ __forceinline__ void build_expert_table_early(ExpertTable &t, const int32_t *offsets, const int32_t *zero, int experts,
                                                         int rows, uint32_t per, int mult, bool each, int32_t *status) {
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass) pdl_wait();
        build_expert_table(t, pass ? offsets : zero, pass ? experts : 0, pass ? rows : 0, per, mult, each, status);
    }
}

// Expert of tile t: the last e with tile[e] <= t (experts without tiles share a
// bound with the next one).
__device__ __forceinline__ int expert_of_tile(const ExpertTable &tab, int experts, int t) {
    int lo = 0, hi = experts - 1;
#pragma unroll 1
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (tab.tile[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// An expert's rows in equal chunks of at most 256, in units of 32: chunks =
// ceil(units / 8), and the smallest size s <= 8 units with s chunks >= units
// (counted instead of divided).  (chunks - 1) s < units, so no chunk is empty.
__device__ __forceinline__ int chunk_rows(int len) {
    const uint32_t units = ((uint32_t)len + 31) / 32, chunks = (units + 7) / 8;
    uint32_t s = 1;
#pragma unroll
    for (uint32_t k = 1; k < 8; ++k) s += k * chunks < units;
    return (int)(s * 32);
}

// A piece of work as the schedule hands it out.
struct __align__(16) ExpertWork {
    int e, m0;       // expert, first index of the M dimension
    int row0, ntok;  // first row; rows of the piece (weight: first column)
    int n;           // MMA width; 0: no more work
    int kb0, kb1;    // k-blocks
    int last;        // weight: valid depth of the last k-block; few-rows kernel: tile number
};
static_assert(sizeof(ExpertWork) == 32, "two 16-byte accesses");

template <int N>
struct ExpertRing {
    ExpertWork work[N];
    uint64_t given[N], taken[N];
    // one thread, before the block's barrier; `readers`: arrivals that free an entry
    __device__ __forceinline__ void init(uint32_t readers) {
        for (int i = 0; i < N; ++i) {
            mbar_init(smem_u32(&given[i]), 1);
            mbar_init(smem_u32(&taken[i]), readers);
        }
    }
    // the schedule's side: waits for entry i to be free, fills it
    __device__ __forceinline__ bool give(uint32_t i, const ExpertWork &w, int64_t budget, volatile int32_t *abort, int32_t *status) {
        const uint32_t r = i % N, ph = (i / N) & 1;
        if (!mbar_wait_bounded(smem_u32(&taken[r]), ph ^ 1, budget, abort, status, kDevTimeoutProducer)) return false;
        work[r] = w;
        mbar_arrive(smem_u32(&given[r]));
        return true;
    }
    // a reader's side; n = 0 at the end or after a wait that ran out
    __device__ __forceinline__ ExpertWork take(uint32_t i, int64_t budget, volatile int32_t *abort, int32_t *status, int32_t code) {
        const uint32_t r = i % N, ph = (i / N) & 1;
        ExpertWork w;
        w.n = 0;
        if (!mbar_wait_bounded(smem_u32(&given[r]), ph, budget, abort, status, code)) return w;
        const int4 *p = reinterpret_cast<const int4 *>(&work[r]);
        const int4 x = p[0], y = p[1];
        w.e = x.x; w.m0 = x.y; w.row0 = x.z; w.ntok = x.w;
        w.n = y.x; w.kb0 = y.y; w.kb1 = y.z; w.last = y.w;
        return w;
    }
    // ... and afterwards, by one thread of each reader
    __device__ __forceinline__ void done(uint32_t i) { mbar_arrive(smem_u32(&taken[i % N])); }
};

}  // namespace cbd
