// experts_stream_sm103.cu -- expert products with few rows per expert
// (serving: single tokens and decode batches), bf16, forward and data:
//   y[i][n]  = sum_k x[i][k]  w[e][n][k]
//   dx[i][k] = sum_n dy[i][n] w[e][n][k]
//
// Every filter that has a row is read once and that read is the time: the floor
// is filter bytes / memory rate.  A tile is 128 of the filter's M dimension x up to
// 16 rows of one expert, which are the MMA's N; its filter comes in blocks of 16 KB
// (64 deep), eleven in flight.
//
// Three tiles for an SM and more: drawn from a counter, each when the loads of the
// one before begin, because the SMs' shares of the memory differ (an even share of
// 107 blocks takes 31 to 42 us).  64 experts of 2048 x 1024, 4 rows each: 45.5 us
// (0.85 of the memory rate; 50 by even shares), 4.5 of them before the first data.
// Drawing the last tiles in pieces of 512 or 1024 deep: 46 to 57, for their joins.
//
// Fewer, or tiles too shallow to hide a draw: cut by filter bytes, the blocks of all
// tiles in one sequence and an equal stretch to each SM.  A tile that lies inside one SM's stretch is stored from there.  A tile cut by a
// stretch's end is joined: each SM writes its fp32 part to the workspace and the
// last of them to arrive (a counter per tile) adds the parts in the order of k
// and stores.  No SM waits for another, and the sum's order is fixed.
//
// Roles: warps 0-3 epilogue, 4 filter loads, 5 MMA and TMEM, 6 row loads, 7
// table and schedule, 8 rows of no expert.  Every wait is bounded.
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

constexpr int RING = 4;

constexpr int BT = kStreamRows;  // rows of a tile
constexpr int S = 11;            // stages
constexpr int A_BYTES = 128 * 64 * 2;
constexpr int B_BYTES = BT * 128;
constexpr int TMEM_COLS = 2 * BT;  // two accumulators
struct Bars {
    ExpertRing<RING> ring;
    uint64_t full[S], empty[S], tfull[2], tempty[2];
    uint32_t tmem;
    int32_t abort, last, vote[8];
    uint64_t want;      // the filter loads took another tile
    uint32_t share[2];  // of the schedule: units of a block, blocks with one more
};
constexpr int SMEM = 1024 + S * (A_BYTES + B_BYTES) + (int)sizeof(ExpertTable) + (int)sizeof(Bars) + 8;
static_assert(SMEM <= 232448, "shared memory of one CTA");
constexpr int THREADS = 9 * 32;

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

// One lane of a warp that runs converged issues; the operands stay warp-uniform.
__device__ __forceinline__ void mma_elect(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// The blocks' equal stretches of `units` things: the first units % g have one more.
struct Share {
    uint32_t each, more;
    __device__ __forceinline__ Share(uint32_t units, uint32_t g) : each(units / g), more(units - each * g) {}
    __device__ __forceinline__ Share(uint32_t each_, uint32_t more_, int) : each(each_), more(more_) {}
    __device__ __forceinline__ uint32_t begin(uint32_t b) const { return b * each + min(b, more); }
    __device__ __forceinline__ uint32_t block_of(uint32_t u) const {
        const uint32_t longer = more * (each + 1);
        return u < longer ? u / (each + 1) : more + (u - longer) / each;
    }
};

template <int DIR>
__global__ void __launch_bounds__(THREADS, 1) experts_stream_kernel(const __grid_constant__ ExpertStreamParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + S * A_BYTES;
    Bars &bars = *reinterpret_cast<Bars *>(sB + S * B_BYTES);
    ExpertTable &tab = *reinterpret_cast<ExpertTable *>(sB + S * B_BYTES + (sizeof(Bars) + 7) / 8 * 8);
    volatile int32_t *abort_flag = &bars.abort;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int mdim = DIR == kExpData ? p.K : p.N, depth = DIR == kExpData ? p.N : p.K;
    const int mt = (mdim + 127) / 128, nkb = (depth + 63) / 64;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 4);
        }
        bars.ring.init(7);
        mbar_init(smem_u32(&bars.want), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(&bars.tmem), TMEM_COLS);
        tc_fence_before();
    }
    if (warp == 4 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.b)) : "memory");
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bars.tmem;
    pdl_next();

    if (warp == 7) {
        build_expert_table_early(tab, p.offsets, &bars.abort, p.experts, p.rows, BT, mt, false, blockIdx.x == 0 ? p.status : nullptr);
        asm volatile("bar.arrive 2, 64;" ::: "memory");
        // ------------------------------------------------------------ schedule
        if (lane == 0) {
            const uint32_t ntiles = (uint32_t)tab.tile[p.experts], g = gridDim.x;
            auto tile = [&](int t, int kb0, int kb1) {
                ExpertWork w;
                w.e = expert_of_tile(tab, p.experts, t);
                const int l = t - tab.tile[w.e], q = l / mt, first = q * BT;
                w.row0 = tab.off[w.e] + first;
                w.ntok = min(BT, tab.len(w.e) - first);
                w.m0 = (l - q * mt) * 128;
                w.n = (w.ntok + 15) & ~15;
                w.kb0 = kb0;
                w.kb1 = kb1;
                w.last = t;
                return w;
            };
            ExpertWork none;
            none.n = 0;
            const bool draw = ntiles >= 3 * g && nkb >= 8;
            for (uint32_t i = 0, t = blockIdx.x; draw; ++i) {
                const ExpertWork w = t < ntiles ? tile((int)t, 0, nkb) : none;
                if (!bars.ring.give(i, w, p.wait_budget, abort_flag, p.status) || w.n == 0) break;
                // the next one once the loads have begun with this one
                if (!mbar_wait_bounded(smem_u32(&bars.want), i & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) break;
                const uint32_t drawn = (uint32_t)atomicAdd(p.drawn, 1);
                // every block draws one too many: ntiles draws in all, and the last one clears
                if (drawn == ntiles - 1) atomicExch(p.drawn, 0);
                t = g + drawn;
            }
            // Cut tiles where their k-blocks spread more evenly over the SMs than whole tiles by more than a join
            // takes: 2.3 us, the time of about eight 16 KB blocks of an SM.
            const uint32_t whole_most = (ntiles + g - 1) / g * nkb, cut_most = (ntiles * nkb + g - 1) / g;
            const uint32_t grain = whole_most <= cut_most + 8 ? nkb : 1;  // k-blocks handed out at a time
            const uint32_t units = ntiles * (grain == 1 ? nkb : 1);
            // no more blocks than units: every block between a tile's first and last has a part of it
            const uint32_t nblocks = max(1u, min(g, units));
            const Share share(units, nblocks);
            bars.share[0] = share.each;
            bars.share[1] = share.more;
            uint32_t u = blockIdx.x < nblocks ? share.begin(blockIdx.x) * grain : 0u;
            const uint32_t hi = blockIdx.x < nblocks ? share.begin(blockIdx.x + 1) * grain : 0u;
            int t = (int)(u / (uint32_t)nkb), kb0 = (int)u - t * nkb;
            for (uint32_t i = 0; !draw; ++i, ++t, kb0 = 0) {
                ExpertWork w = none;
                if (u < hi) {
                    w = tile(t, kb0, (int)min((uint32_t)nkb, (uint32_t)kb0 + (hi - u)));
                    u += (uint32_t)(w.kb1 - kb0);
                }
                if (!bars.ring.give(i, w, p.wait_budget, abort_flag, p.status) || w.n == 0) break;
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        pdl_wait();
        asm volatile("bar.sync 2, 64;" ::: "memory");  // the table
        // ------------------------------------------------------------ rows of no expert: zeros
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
        const int lo = tab.off[0], hi = tab.off[p.experts], vec = mdim / 8;
        const int64_t nfill = (int64_t)lo + (p.rows - hi);
        const bool lines = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)p.ldo * 2) & 15) == 0;
        for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
            __nv_bfloat16 *row = out + (f < lo ? f : hi + (f - lo)) * p.ldo;
            if (lines)
                for (int c = lane; c < vec; c += 32) reinterpret_cast<uint4 *>(row)[c] = make_uint4(0u, 0u, 0u, 0u);
            else
                for (int c = lane; c < mdim; c += 32) row[c] = __nv_bfloat16(0.f);
        }
    } else if (warp == 4 || warp == 6) {
        // ------------------------------------------------------------ loads
        pdl_wait();
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (uint32_t i = 0; ok; ++i) {
                const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                if (w.n == 0) break;
                bars.ring.done(i);
                if (warp == 4) mbar_arrive(smem_u32(&bars.want));
                for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % S, ph = (it / S) & 1, bar = full0 + 8 * s;
                    if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    if (warp == 4) {
                        mbar_arrive_expect_tx(bar, A_BYTES + B_BYTES);
                        const uint32_t dst = smem_u32(sA + s * A_BYTES);
                        if constexpr (DIR == kExpForward) {
                            load_3d(dst, &p.a, bar, kb * 64, w.m0, w.e);
                        } else {
                            load_3d(dst, &p.a, bar, w.m0, kb * 64, w.e);
                            load_3d(dst + 8192, &p.a, bar, w.m0 + 64, kb * 64, w.e);
                        }
                    } else {
                        load_2d(smem_u32(sB + s * B_BYTES), &p.b, bar, kb * 64, w.row0);
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
        pdl_wait();
        constexpr bool A_K = DIR == kExpForward;
        constexpr uint32_t A_STEP = A_K ? 2 : 128;
        const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((A_K ? 0u : 1u) << 15) | ((uint32_t)(128 >> 4) << 24);
        const uint64_t a_desc0 = smem_desc_sw128(smem_u32(sA), A_K ? 16 : 8192, 1024);
        const uint64_t b_desc0 = smem_desc_sw128(smem_u32(sB), 16, 1024);
        const uint32_t a_lo = (uint32_t)a_desc0, a_hi = (uint32_t)(a_desc0 >> 32), b_lo = (uint32_t)b_desc0, b_hi = (uint32_t)(b_desc0 >> 32);
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (uint32_t use = 0; ok; ++use) {
            ExpertWork w = bars.ring.take(use, p.wait_budget, abort_flag, p.status, kDevTimeoutMma);
            w.n = __shfl_sync(0xffffffffu, w.n, 0);
            const int count = __shfl_sync(0xffffffffu, w.kb1 - w.kb0, 0);
            if (w.n == 0) break;
            if (lane == 0) bars.ring.done(use);
            const uint32_t b = use & 1, bph = (use >> 1) & 1;
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(tempty0 + 8 * b, bph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
            if (!ok) break;
            tc_fence_after();
            const uint32_t id = idesc0 | ((uint32_t)(w.n >> 3) << 17), d = tmem_base + b * BT;
            uint32_t acc = 0;
            for (int left = count; left > 0; --left) {
                ok = __all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                if (!ok) break;
                const uint32_t ad = a_lo + s * (A_BYTES >> 4), bd = b_lo + s * (B_BYTES >> 4);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    mma_elect(d, ad + A_STEP * kk, a_hi, bd + 2 * kk, b_hi, id, acc);
                    acc = 1;
                }
                commit_elect(empty0 + 8 * s);
                if (++s == (uint32_t)S) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (ok) commit_elect(tfull0 + 8 * b);
        }
        if (!ok) {
            for (int q = 0; q < 100; ++q) __nanosleep(1000);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ epilogue
        pdl_wait();
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
        const uint32_t lane_base = tmem_base + ((uint32_t)(warp * 32) << 16);
        bool ok = true;  // after a wait that ran out: no stores, but every barrier and counter as usual
        for (uint32_t use = 0;; ++use) {
            const ExpertWork w = bars.ring.take(use, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            bool more = __all_sync(0xffffffffu, w.n != 0);
            if (more && lane == 0) bars.ring.done(use);
            // the four warps meet at barriers below: they go on or stop together
            volatile int32_t *vote = bars.vote + (use & 1) * 4;
            if (lane == 0) vote[warp] = more;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (!(vote[0] & vote[1] & vote[2] & vote[3])) break;
            const uint32_t b = use & 1;
            if (ok) ok = mbar_wait_bounded(tfull0 + 8 * b, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            const bool whole = w.kb0 == 0 && w.kb1 == nkb;
            const int m = w.m0 + (int)threadIdx.x;
            __nv_bfloat16 *dst = out + (int64_t)w.row0 * p.ldo + m;
            float *slot = p.parts + ((int64_t)blockIdx.x * 2 + (w.kb0 == 0 ? 1 : 0)) * (BT * 128) + threadIdx.x;
            uint32_t v[BT];
            tmem_ld16(lane_base + b * BT, v);
#pragma unroll
            for (int q = 0; q < BT; ++q) {
                if (q >= w.ntok) break;
                if (whole) {
                    if (ok && m < mdim) dst[(int64_t)q * p.ldo] = __float2bfloat16_rn(__uint_as_float(v[q]));
                } else {
                    __stcg(slot + q * 128, __uint_as_float(v[q]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty0 + 8 * b);
            if (whole) continue;

            const uint32_t first = (uint32_t)w.last * nkb;  // (grain 1)
            const Share share(bars.share[0], bars.share[1], 0);
            const int c0 = (int)share.block_of(first), c1 = (int)share.block_of(first + nkb - 1);
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
                float a[BT];
#pragma unroll
                for (int q = 0; q < BT; ++q) a[q] = 0.f;
                for (int c = c0; c <= c1; ++c) {
                    const float *part = p.parts + ((int64_t)c * 2 + (c == c0 ? 1 : 0)) * (BT * 128) + threadIdx.x;
                    float x[BT];
#pragma unroll
                    for (int q = 0; q < BT; ++q) x[q] = q < w.ntok ? __ldcg(part + q * 128) : 0.f;
#pragma unroll
                    for (int q = 0; q < BT; ++q) a[q] += x[q];
                }
#pragma unroll
                for (int q = 0; q < BT; ++q)
                    if (ok && q < w.ntok && m < mdim) dst[(int64_t)q * p.ldo] = __float2bfloat16_rn(a[q]);
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");  // bars.last is written again
        }
    }

    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <int DIR>
cudaError_t launch_dir(const ExpertStreamParams &p, int grid, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_stream_kernel<DIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(experts_stream_kernel<DIR>, grid, THREADS, SMEM, s, p);
}

}  // namespace

cudaError_t launch_experts_stream(const ExpertStreamParams &p, int dir, int grid, cudaStream_t s) {
    return dir == kExpForward ? launch_dir<kExpForward>(p, grid, s) : launch_dir<kExpData>(p, grid, s);
}

}  // namespace cbd
