// experts_stream_sm103.cu -- expert products with few rows per expert
// (serving: single tokens and decode batches), bf16, forward and data:
//   y[i][n]  = sum_k x[i][k]  w[e][n][k]
//   dx[i][k] = sum_n dy[i][n] w[e][n][k]
//
// Every filter that has a row is read once and that read is the time: the floor
// is filter bytes / memory rate.  So the work is cut by filter bytes, not by
// tiles: the 16 KB blocks (128 of the filter's M dimension x 64 deep) of all
// tiles in one sequence, an equal stretch to each SM, eight to eleven blocks in
// flight.  A tile is 128 x up to BT rows of one expert; the rows are the MMA's N
// (steps of 16), so one row costs 16 columns.
//
// A tile that lies inside one SM's stretch is stored from there.  A tile cut by a
// stretch's end is joined: each SM writes its fp32 part to the workspace and the
// last of them to arrive (a counter per tile) adds the parts in the order of k
// and stores.  No SM waits for another, and the sum's order is fixed.
//
// Roles: warps 0-3 epilogue, 4 filter loads, 5 MMA and TMEM, 6 row loads.
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "device_util.cuh"
#include "expert_table.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "train.h"

namespace cbd {

namespace {

template <int BT>
struct Cfg {
    static constexpr int S = BT == 16 ? 11 : 8;  // stages
    static constexpr int A_BYTES = 128 * 64 * 2;
    static constexpr int B_BYTES = BT * 128;
    static constexpr int TMEM_COLS = 2 * BT;  // two accumulators (32 or 128 columns)
    struct Bars {
        uint64_t full[S], empty[S], tfull[2], tempty[2];
        uint32_t tmem;
        int32_t abort, last;
    };
    static constexpr int SMEM = 1024 + S * (A_BYTES + B_BYTES) + (int)sizeof(ExpertTable) + (int)sizeof(Bars) + 8;
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};
constexpr int THREADS = 7 * 32;

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// A block's stretch of the sequence (tile, k-block), tile by tile.
struct Stretch {
    int64_t u, hi;
    int nkb;
    int t, kb0, kb1;  // current segment
    __device__ __forceinline__ Stretch(int64_t units, int nkb_, int b, int g) : nkb(nkb_) {
        u = units * b / g;
        hi = b < g ? units * (b + 1) / g : u;
    }
    __device__ __forceinline__ bool next() {
        if (u >= hi) return false;
        t = (int)(u / nkb);
        kb0 = (int)(u - (int64_t)t * nkb);
        kb1 = (int)min((int64_t)nkb, kb0 + (hi - u));
        u += kb1 - kb0;
        return true;
    }
};
// block whose stretch holds unit u
__device__ __forceinline__ int block_of(int64_t u, int64_t units, int g) { return (int)(((u + 1) * g - 1) / units); }

template <int DIR, int BT>
__global__ void __launch_bounds__(THREADS, 1) experts_stream_kernel(const __grid_constant__ ExpertStreamParams p) {
    using C = Cfg<BT>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + S * C::A_BYTES;
    typename C::Bars &bars = *reinterpret_cast<typename C::Bars *>(sB + S * C::B_BYTES);
    ExpertTable &tab = *reinterpret_cast<ExpertTable *>(sB + S * C::B_BYTES + (sizeof(typename C::Bars) + 7) / 8 * 8);
    volatile int32_t *abort_flag = &bars.abort;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int mdim = DIR == kExpData ? p.K : p.N, depth = DIR == kExpData ? p.N : p.K;
    const int mt = (mdim + 127) / 128, nkb = (depth + 63) / 64;

    load_expert_offsets(tab, p.offsets, p.experts);
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 4);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(&bars.tmem), C::TMEM_COLS);
        tc_fence_before();
    }
    if (warp == 4 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.b)) : "memory");
    }
    __syncthreads();
    if (warp == 0)
        build_expert_table(tab, p.experts, p.rows, BT, mt, kTilesInOrder, blockIdx.x == 0 ? p.status : nullptr);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars.tmem;
    const int64_t units = (int64_t)tab.tile[p.experts] * nkb;
    // no more blocks than units: every block between a tile's first and last has a part of it
    const int nblocks = (int)min((int64_t)gridDim.x, max(units, (int64_t)1));
    Stretch seg(units, nkb, min((int)blockIdx.x, nblocks), nblocks);

    // rows and M block of tile t
    struct Where {
        int e, row0, ntok, m0;
    };
    auto where = [&](int t) {
        Where w;
        w.e = position_of_tile(tab, p.experts, t);
        const int l = t - tab.tile[w.e], len = tab.len(w.e), first = (l / mt) * BT;
        w.row0 = tab.off[w.e] + first;
        w.ntok = min(BT, len - first);
        w.m0 = (l % mt) * 128;
        return w;
    };

    if (warp == 4 || warp == 6) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            while (ok && seg.next()) {
                const Where w = where(seg.t);
                for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++it) {
                    const uint32_t s = it % S, ph = (it / S) & 1, bar = full0 + 8 * s;
                    if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (warp == 4) {
                        mbar_arrive_expect_tx(bar, C::A_BYTES + C::B_BYTES);
                        const uint32_t dst = smem_u32(sA + s * C::A_BYTES);
                        if constexpr (DIR == kExpForward) {
                            load_3d(dst, &p.a, bar, kb * 64, w.m0, w.e);
                        } else {
                            load_3d(dst, &p.a, bar, w.m0, kb * 64, w.e);
                            load_3d(dst + 8192, &p.a, bar, w.m0 + 64, kb * 64, w.e);
                        }
                    } else {
                        load_2d(smem_u32(sB + s * C::B_BYTES), &p.b, bar, kb * 64, w.row0);
                    }
                }
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            constexpr bool A_K = DIR == kExpForward;
            constexpr uint32_t A_STEP = A_K ? 2 : 128;
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((A_K ? 0u : 1u) << 15) | ((uint32_t)(128 >> 4) << 24);
            const uint64_t a_desc0 = smem_desc_sw128(smem_u32(sA), A_K ? 16 : 8192, 1024);
            const uint64_t b_desc0 = smem_desc_sw128(smem_u32(sB), 16, 1024);
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t use = 0; ok && seg.next(); ++use) {
                const Where w = where(seg.t);
                const uint32_t b = use & 1, bph = (use >> 1) & 1;
                if (!mbar_wait_bounded(tempty0 + 8 * b, bph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t id = idesc0 | ((uint32_t)(((w.ntok + 15) & ~15) >> 3) << 17), d = tmem_base + b * BT;
                for (int kb = seg.kb0; kb < seg.kb1; ++kb, ++it) {
                    const uint32_t s = it % S, ph = (it / S) & 1;
                    if (!mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    const uint64_t ad = a_desc0 + (uint64_t)((s * C::A_BYTES) >> 4), bd = b_desc0 + (uint64_t)((s * C::B_BYTES) >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) tc_mma(d, ad + A_STEP * kk, bd + 2 * kk, id, (kb != seg.kb0 || kk != 0) ? 1u : 0u);
                    tc_commit(empty0 + 8 * s);
                }
                if (ok) tc_commit(tfull0 + 8 * b);
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
        {
            // rows of no expert: zeros
            const int lo = tab.off[0], hi = tab.off[p.experts], vec = mdim / 8;
            const int64_t nfill = (int64_t)lo + (p.rows - hi);
            for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
                uint4 *row = reinterpret_cast<uint4 *>(out + (f < lo ? f : hi + (f - lo)) * p.ldo);
                for (int c = threadIdx.x; c < vec; c += 128) row[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        const uint32_t lane_base = tmem_base + ((uint32_t)(warp * 32) << 16);
        bool ok = true;  // after a wait that ran out: no stores, but every barrier and counter as usual
        for (uint32_t use = 0; seg.next(); ++use) {
            const Where w = where(seg.t);
            const uint32_t b = use & 1;
            if (ok) ok = mbar_wait_bounded(tfull0 + 8 * b, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const bool whole = seg.kb0 == 0 && seg.kb1 == nkb;
            const int m = w.m0 + (int)threadIdx.x;
            __nv_bfloat16 *dst = out + (int64_t)w.row0 * p.ldo + m;
            float *slot = p.parts + ((int64_t)blockIdx.x * 2 + (seg.kb0 == 0 ? 1 : 0)) * (BT * 128) + threadIdx.x;
            constexpr int G = BT < 32 ? BT : 32;
#pragma unroll 1
            for (int g = 0; g < w.ntok; g += G) {
                uint32_t v[G];
                if constexpr (G == 16)
                    tmem_ld16(lane_base + b * BT + g, v);
                else
                    tmem_ld32(lane_base + b * BT + g, v);
#pragma unroll
                for (int q = 0; q < G; ++q) {
                    if (g + q >= w.ntok) break;
                    if (whole) {
                        if (ok && m < mdim) dst[(int64_t)(g + q) * p.ldo] = __float2bfloat16_rn(__uint_as_float(v[q]));
                    } else {
                        __stcg(slot + (g + q) * 128, __uint_as_float(v[q]));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty0 + 8 * b);
            if (whole) continue;

            const int64_t first = (int64_t)seg.t * nkb;
            const int c0 = block_of(first, units, nblocks), c1 = block_of(first + nkb - 1, units, nblocks);
            __threadfence();
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (threadIdx.x == 0) {
                const int n = atomicAdd(p.arrived + c0, 1);
                bars.last = n == c1 - c0;
                if (n == c1 - c0) p.arrived[c0] = 0;
                __threadfence();
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (*(volatile int32_t *)&bars.last) {
                __threadfence();
#pragma unroll 1
                for (int g = 0; g < w.ntok; g += 16) {
                    float a[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) a[q] = 0.f;
                    for (int c = c0; c <= c1; ++c) {
                        const float *part = p.parts + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * (BT * 128) + threadIdx.x;
                        float x[16];
#pragma unroll
                        for (int q = 0; q < 16; ++q) x[q] = g + q < w.ntok ? __ldcg(part + (g + q) * 128) : 0.f;
#pragma unroll
                        for (int q = 0; q < 16; ++q) a[q] += x[q];
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        if (ok && g + q < w.ntok && m < mdim) dst[(int64_t)(g + q) * p.ldo] = __float2bfloat16_rn(a[q]);
                }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");  // bars.last is written again
        }
    }

    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem_base, C::TMEM_COLS);
    }
}

template <int DIR, int BT>
cudaError_t launch_bt(const ExpertStreamParams &p, int grid, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_stream_kernel<DIR, BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<BT>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    experts_stream_kernel<DIR, BT><<<grid, THREADS, Cfg<BT>::SMEM, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_experts_stream(const ExpertStreamParams &p, int dir, int bt, int grid, cudaStream_t s) {
    if (dir == kExpForward) return bt == 16 ? launch_bt<kExpForward, 16>(p, grid, s) : launch_bt<kExpForward, 64>(p, grid, s);
    return bt == 16 ? launch_bt<kExpData, 16>(p, grid, s) : launch_bt<kExpData, 64>(p, grid, s);
}

}  // namespace cbd
