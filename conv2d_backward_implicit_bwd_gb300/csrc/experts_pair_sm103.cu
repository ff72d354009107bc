// experts_pair_sm103.cu -- matrix products grouped by expert on pairs of SMs
// (tcgen05 cta_group::2, bf16 operands, fp32 accumulation).
//
//   forward  y[i][n]     = sum_k x[i][k]  w[e][n][k]
//   data     dx[i][k]    = sum_n dy[i][n] w[e][n][k]
//   weight   dw[e][n][k] (+)= sum_{i in e} dy[i][n] x[i][k]
//
// Orientation.  The filter's dimension is the MMA's M (256 per pair, 128 per
// CTA) and an expert's rows are its N, which the instruction takes in steps of
// 32: an expert of 70 rows costs a 96-wide product instead of a 256-high one.
// So forward and data compute the transposed tile D[n][i] and the epilogue
// turns it around in shared memory.  weight has both dimensions fixed and the
// ragged one as contraction: D[n][k], rows in blocks of 64.
//
//            A (M)                       B (N)                     contraction
//   forward  w rows n, K-major           x rows i, K-major         k
//   data     w columns k, MN-major       dy rows i, K-major        n
//   weight   dy columns n, MN-major      x columns k, MN-major     i
//
// A tile has up to 512 columns of B in two halves of up to 256, each with its
// own 256 TMEM columns ("slot").  Slots are used in turn by the halves of all
// tiles, so that a one-half tile is double-buffered against the next and a
// two-half tile's successor starts on the first half while the epilogue drains
// the second.  A two-half tile moves 48 KB per CTA for each 64-deep step of
// 1024 MMA clocks, a one-half tile 32 KB for 512: the operands come from L2 at
// about 45 bytes per SM clock, so wide tiles run nearer the MMA rate and narrow
// ones spread over more pairs.
//
// Ragged ends.  Rows past an expert's end that a box brings along are other
// columns of D (forward, data), never stored.  For weight they would be
// summed: the last block multiplies only its valid 16-row steps, and where the
// last step is partial a helper warp of each CTA zeroes its rows in shared
// memory after they have landed (both operands: 0 x NaN is NaN) before the MMA
// may read them.
//
// Roles per CTA: warps 0-3 epilogue, 4 A loads, 5 MMA (leader CTA) and TMEM,
// 6-7 B loads (one half each), 8 helper of weight's last blocks.  Persistent over the
// tiles of all experts; every wait is bounded.
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

constexpr int S = 4;  // pipeline stages
constexpr int A_BYTES = 128 * 64 * 2;
constexpr int HALF_BYTES = 128 * 64 * 2;  // one half's B rows (or columns) of one CTA
constexpr int B_BYTES = 2 * HALF_BYTES;
constexpr int OUT_BYTES = 16384;  // epilogue staging
constexpr int THREADS = 9 * 32;

struct Bars {
    uint64_t full[S], empty[S];
    uint64_t tail[S], peer[S];  // weight: last blocks landed in this CTA; peer's rows zeroed
    uint64_t tfull[2], tempty[2];
    uint32_t tmem;
    int32_t abort;
};
constexpr int SMEM = 1024 + S * (A_BYTES + B_BYTES) + OUT_BYTES + (int)sizeof(ExpertTable) + (int)sizeof(Bars);
static_assert(SMEM <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// (bar in this CTA)
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ bool test_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// One tile: the same for every role.
struct Tile {
    int e, m0;          // expert, first row of the M dimension
    int row0, ntok;     // forward, data: first row, rows of the tile
    int c0;             // weight: first column
    int halves;         // 0: weight tile of an expert without rows
    int n0, n1;         // MMA width of each half
    int at1;            // first row (column) of the second half within the tile
    int nkb, last;      // k-blocks, valid depth of the last one
};

template <int DIR>
__device__ __forceinline__ Tile tile_of(const ExpertPairParams &p, const ExpertTable &tab, int mt, int nt, int t) {
    Tile r;
    if constexpr (DIR == kExpWeight) {
        r.e = t / (mt * nt);
        const int l = t - r.e * mt * nt;
        r.m0 = (l % mt) * 256;
        r.c0 = (l / mt) * p.wide;
        r.row0 = tab.off[r.e];
        const int len = tab.len(r.e);
        r.nkb = (len + 63) / 64;
        r.last = len - (r.nkb - 1) * 64;
        r.halves = len == 0 ? 0 : (p.wide > 256 && r.c0 + 256 < p.K) ? 2 : 1;
        r.n0 = r.n1 = 256;
        r.at1 = 256;
        r.ntok = 0;
    } else {
        r.e = expert_of_tile(tab, p.experts, t);
        const int l = t - tab.tile[r.e], len = tab.len(r.e);
        r.m0 = (l % mt) * 256;
        // an expert's rows in equal chunks, a chunk in equal halves, rounded up to 32
        const int chunks = (len + p.wide - 1) / p.wide;
        const int size = ((len + chunks - 1) / chunks + 31) & ~31;
        const int first = (l / mt) * size;
        r.row0 = tab.off[r.e] + first;
        r.ntok = min(size, len - first);
        r.halves = r.ntok > 256 ? 2 : 1;
        r.n0 = r.halves == 2 ? ((r.ntok + 1) / 2 + 31) & ~31 : (r.ntok + 31) & ~31;
        r.at1 = r.n0;
        r.n1 = r.halves == 2 ? (r.ntok - r.n0 + 31) & ~31 : 0;
        const int depth = DIR == kExpForward ? p.K : p.N;
        r.nkb = (depth + 63) / 64;
        r.last = 64;  // past the depth both operands read as zero
        r.c0 = 0;
    }
    return r;
}

template <int DIR>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) experts_pair_kernel(const __grid_constant__ ExpertPairParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + S * A_BYTES;
    uint8_t *stage = sB + S * B_BYTES;
    ExpertTable &tab = *reinterpret_cast<ExpertTable *>(stage + OUT_BYTES);
    Bars &bars = *reinterpret_cast<Bars *>(stage + OUT_BYTES + sizeof(ExpertTable));
    static_assert(sizeof(ExpertTable) % 8 == 0, "barriers on 8 bytes");
    volatile int32_t *abort_flag = &bars.abort;

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tail0 = smem_u32(bars.tail),
                   peer0 = smem_u32(bars.peer), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int mdim = DIR == kExpData ? p.K : p.N;
    const int mt = (mdim + 255) / 256;
    const int nt = DIR == kExpWeight ? (p.K + p.wide - 1) / p.wide : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(tail0 + 8 * s, 1);
            mbar_init(peer0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 8);  // 4 epilogue warps of each CTA
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 5) {
        tmem_alloc2(smem_u32(&bars.tmem), 512);
        tc_fence_before();
    }
    if (warp == 4 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.b)) : "memory");
    }
    if (warp == 0)
        build_expert_table(tab, p.offsets, p.experts, p.rows, p.wide, mt, blockIdx.x == 0 ? p.status : nullptr);
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = bars.tmem;
    if (threadIdx.x == 0 && !leader) {
        // the pair's MMAs write this CTA's rows at the leader's TMEM address
        if (ld_shared_cluster_u32(mapa_shared(smem_u32(&bars.tmem), 0)) != tmem_base) record_status(p.status, kDevFaultIndex);
    }
    const int total = DIR == kExpWeight ? p.experts * mt * nt : tab.tile[p.experts];

    if (warp == 4 || warp == 6 || warp == 7) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            const uint32_t full_leader0 = mapa_shared(full0, 0);
            const int h = warp - 6;  // B half of this warp
            uint32_t it = 0;
            bool ok = true, issued = false;
            for (int t = pair; t < total && ok; t += npairs) {
                const Tile w = tile_of<DIR>(p, tab, mt, nt, t);
                const int half_rows = DIR == kExpWeight ? 128 : (h == 1 ? w.n1 : w.n0) / 2;
                const int half_at = h == 1 ? w.at1 : 0;
                const int boxes0 = DIR == kExpWeight ? 2 : (w.n0 / 2 + 63) / 64;
                const int boxes1 = w.halves < 2 ? 0 : DIR == kExpWeight ? 2 : (w.n1 / 2 + 63) / 64;
                const uint32_t bytes = (uint32_t)A_BYTES + 8192u * (uint32_t)(boxes0 + boxes1);  // of one CTA
                const int my_boxes = h == 0 ? boxes0 : h == 1 ? boxes1 : 0;
                for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                    const uint32_t s = it % S, ph = (it / S) & 1;
                    if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                        ok = false;
                        break;
                    }
                    // weight: a partial last step goes through the helper warp, on this CTA's own barrier
                    const bool fix = DIR == kExpWeight && kb == w.nkb - 1 && (w.last & 15) != 0;
                    const uint32_t bar = fix ? tail0 + 8 * s : full_leader0 + 8 * s;
                    if (warp == 4) {
                        if (fix)
                            mbar_arrive_expect_tx(tail0 + 8 * s, bytes);
                        else if (leader)
                            mbar_arrive_expect_tx(full0 + 8 * s, 2 * bytes);
                        const uint32_t dst = smem_u32(sA + s * A_BYTES);
                        const int m = w.m0 + (int)rank * 128;
                        if constexpr (DIR == kExpForward) {
                            tma_load_3d_pair(dst, &p.a, bar, kb * 64, m, w.e);
                        } else if constexpr (DIR == kExpData) {
                            tma_load_3d_pair(dst, &p.a, bar, m, kb * 64, w.e);
                            tma_load_3d_pair(dst + 8192, &p.a, bar, m + 64, kb * 64, w.e);
                        } else {
                            for (int q = 0; q < 2; ++q)
                                if (fix)
                                    tma_load_2d(dst + 8192 * q, &p.a, bar, m + 64 * q, w.row0 + kb * 64);
                                else
                                    tma_load_2d_pair(dst + 8192 * q, &p.a, bar, m + 64 * q, w.row0 + kb * 64);
                        }
                    } else {
                        const uint32_t dst = smem_u32(sB + s * B_BYTES + h * HALF_BYTES);
                        for (int q = 0; q < my_boxes; ++q) {
                            const int at = half_at + (int)rank * half_rows + 64 * q;
                            if constexpr (DIR == kExpWeight) {
                                if (fix)
                                    tma_load_2d(dst + 8192 * q, &p.b, bar, w.c0 + at, w.row0 + kb * 64);
                                else
                                    tma_load_2d_pair(dst + 8192 * q, &p.b, bar, w.c0 + at, w.row0 + kb * 64);
                            } else {
                                tma_load_2d_pair(dst + 8192 * q, &p.b, bar, kb * 64, w.row0 + at);
                            }
                        }
                    }
                    issued = true;
                }
            }
            if (!ok && issued) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA (leader)
        if (leader && lane == 0) {
            constexpr bool A_K = DIR == kExpForward, B_K = DIR != kExpWeight;
            constexpr uint32_t A_STEP = A_K ? 2 : 128, B_STEP = B_K ? 2 : 128;  // a 16-deep step, in 16 bytes
            const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((A_K ? 0u : 1u) << 15) | ((B_K ? 0u : 1u) << 16) | ((uint32_t)(256 >> 4) << 24);
            const uint64_t a_desc0 = smem_desc_sw128(smem_u32(sA), A_K ? 16 : 8192, 1024);
            const uint64_t b_desc0 = smem_desc_sw128(smem_u32(sB), B_K ? 16 : 8192, 1024);
            uint32_t it = 0, use = 0;  // stages and slots used so far
            bool ok = true, issued = false;
            for (int t = pair; t < total && ok; t += npairs) {
                const Tile w = tile_of<DIR>(p, tab, mt, nt, t);
                if (w.halves == 0) continue;
                const uint32_t s0 = use & 1, p0 = ((use >> 1) & 1) ^ 1;
                const uint32_t s1 = s0 ^ 1, p1 = (((use + 1) >> 1) & 1) ^ 1;
                if (!mbar_wait_bounded(tempty0 + 8 * s0, p0, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t id0 = idesc0 | ((uint32_t)(w.n0 >> 3) << 17), id1 = idesc0 | ((uint32_t)(w.n1 >> 3) << 17);
                const uint32_t d0 = tmem_base + s0 * 256, d1 = tmem_base + s1 * 256;
                const uint32_t it0 = it;
                int pend = 0;  // first k-block whose second half is pending
                bool h1 = false;
                const bool two = w.halves == 2;
                auto steps = [&](int kb) { return DIR == kExpWeight && kb == w.nkb - 1 ? (w.last + 15) / 16 : 4; };
                auto second = [&](int kb) {
                    const uint32_t sq = (it0 + (uint32_t)kb) % S;
                    const uint64_t ad = a_desc0 + (uint64_t)((sq * A_BYTES) >> 4);
                    const uint64_t bd = b_desc0 + (uint64_t)((sq * B_BYTES + HALF_BYTES) >> 4);
                    const int n = steps(kb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < n) tc_mma2(d1, ad + A_STEP * kk, bd + B_STEP * kk, id1, (kb | kk) != 0 ? 1u : 0u);
                    tc_commit2_mc(empty0 + 8 * sq, (uint16_t)0x3);
                };
                for (int kb = 0; kb < w.nkb; ++kb, ++it) {
                    const uint32_t s = it % S, ph = (it / S) & 1;
                    if (!mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                        ok = false;
                        break;
                    }
                    const uint64_t ad = a_desc0 + (uint64_t)((s * A_BYTES) >> 4), bd = b_desc0 + (uint64_t)((s * B_BYTES) >> 4);
                    const int n = steps(kb);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (kk < n) tc_mma2(d0, ad + A_STEP * kk, bd + B_STEP * kk, id0, (kb | kk) != 0 ? 1u : 0u);
                    issued = true;
                    if (!two) {
                        tc_commit2_mc(empty0 + 8 * s, (uint16_t)0x3);
                        continue;
                    }
                    if (!h1) {
                        h1 = test_wait(tempty0 + 8 * s1, p1);
                        if (!h1 && kb + 1 - pend >= S) {  // every stage is held for the second half
                            if (!mbar_wait_bounded(tempty0 + 8 * s1, p1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                                ok = false;
                                break;
                            }
                            h1 = true;
                        }
                        if (h1) tc_fence_after();
                    }
                    if (h1)
                        for (; pend <= kb; ++pend) second(pend);
                }
                if (!ok) break;
                tc_commit2_mc(tfull0 + 8 * s0, (uint16_t)0x3);
                if (two) {
                    if (pend < w.nkb) {
                        if (!mbar_wait_bounded(tempty0 + 8 * s1, p1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        for (; pend < w.nkb; ++pend) second(pend);
                    }
                    tc_commit2_mc(tfull0 + 8 * s1, (uint16_t)0x3);
                }
                use += (uint32_t)w.halves;
            }
            if (!ok && issued) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else if (warp == 8) {
        // ------------------------------------------------------------ weight: rows past the expert's end
        if constexpr (DIR == kExpWeight) {
            uint32_t it = 0, phase = 0;  // bit s: parity of the next use of tail[s] and peer[s]
            for (int t = pair; t < total; t += npairs) {
                const Tile w = tile_of<DIR>(p, tab, mt, nt, t);
                it += (uint32_t)w.nkb;
                if (w.nkb == 0 || (w.last & 15) == 0) continue;
                const uint32_t s = (it - 1) % S, ph = (phase >> s) & 1;
                phase ^= 1u << s;
                bool ok = mbar_wait_bounded(tail0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                if (!__all_sync(0xffffffffu, ok)) break;
                // rows [last, next multiple of 16) of each 64 x 64 block: whole 128-byte lines, so the swizzle
                // within a line does not matter
                const int lo = w.last, n = ((lo + 15) & ~15) - lo;
                const int blocks = 2 + 2 * w.halves;
                for (int i = lane; i < blocks * n * 8; i += 32) {
                    const int blk = i / (n * 8), r = i / 8 % n, c = i % 8;
                    uint8_t *base = blk < 2 ? sA + s * A_BYTES + blk * 8192 : sB + s * B_BYTES + (blk - 2) * 8192;
                    *reinterpret_cast<uint4 *>(base + (lo + r) * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (!leader) {
                        mbar_arrive_remote(mapa_shared(peer0 + 8 * s, 0));
                    } else {
                        ok = mbar_wait_bounded(peer0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                        asm volatile("fence.acq_rel.cluster;" ::: "memory");
                        if (ok) mbar_arrive(full0 + 8 * s);
                    }
                }
                if (!__all_sync(0xffffffffu, ok)) break;
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (both CTAs)
        const uint32_t tempty_leader0 = mapa_shared(tempty0, 0);
        const uint32_t lane_base = tmem_base + ((uint32_t)(warp * 32) << 16);
        uint32_t use = 0;
        if constexpr (DIR != kExpWeight) {
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
            // rows of no expert: zeros (16-byte stores; the width is a multiple of 8)
            const int lo = tab.off[0], hi = tab.off[p.experts], vec = mdim / 8;
            const int64_t nfill = (int64_t)lo + (p.rows - hi);
            for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
                uint4 *row = reinterpret_cast<uint4 *>(out + (f < lo ? f : hi + (f - lo)) * p.ldo);
                for (int c = threadIdx.x; c < vec; c += 128) row[c] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        uint32_t buf = 0;
        bool ok = true;
        for (int t = pair; t < total; t += npairs) {
            const Tile w = tile_of<DIR>(p, tab, mt, nt, t);
            const int m = w.m0 + (int)rank * 128;
            if constexpr (DIR == kExpWeight) {
                // 32 x 32 fp32 pieces (a warp's rows, 128 bytes each) through swizzled staging and TMA stores,
                // added in L2 when accumulating: one writer per element, so the order is fixed
                const int halves = w.halves ? w.halves : (p.accumulate ? 0 : (p.wide > 256 && w.c0 + 256 < p.K) ? 2 : 1);
                const int mrow = m + warp * 32;
                uint8_t *slab = stage + warp * 4096;
                for (int h = 0; h < halves; ++h) {
                    const uint32_t slot = use & 1;
                    if (w.halves) {
                        ok = mbar_wait_bounded(tfull0 + 8 * slot, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                        if (!__all_sync(0xffffffffu, ok)) break;
                        tc_fence_after();
                    }
                    const int c0 = w.c0 + (h ? w.at1 : 0);
#pragma unroll 1
                    for (int g = 0; g < 8; ++g) {
                        uint32_t v[32];
                        if (w.halves) {
                            tmem_ld32(lane_base + slot * 256 + g * 32, v);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = 0u;
                        }
                        if (lane == 0) bulk_wait_read();
                        __syncwarp();
                        const uint32_t sb = smem_u32(slab) + (uint32_t)lane * 128u;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (((uint32_t)q ^ (lane & 7)) << 4)),
                                         "r"(v[4 * q]), "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3])
                                         : "memory");
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0 && mrow < p.N && c0 + g * 32 < p.K) {
                            const uint64_t map = reinterpret_cast<uint64_t>(&p.o);
                            if (p.accumulate)
                                asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                                             "r"(c0 + g * 32), "r"(mrow), "r"(w.e), "r"(smem_u32(slab))
                                             : "memory");
                            else
                                asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                                             "r"(c0 + g * 32), "r"(mrow), "r"(w.e), "r"(smem_u32(slab))
                                             : "memory");
                            bulk_commit();
                        }
                    }
                    if (w.halves) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_remote(tempty_leader0 + 8 * slot);
                        ++use;
                    }
                }
            } else {
                // columns of the accumulator are rows of the output: 32 of them at a time are turned around in
                // shared memory ([row][128 of the M dimension], 256 bytes) and leave in 16-byte stores, two
                // whole row segments to an instruction.  (A bulk copy per row took 95 clocks each: 25 us a tile.)
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
                const int col = (lane & 15) * 8;
                const bool col_ok = m + col < mdim;
                for (int h = 0; h < w.halves; ++h, ++use) {
                    const uint32_t slot = use & 1;
                    // after a wait that ran out the warps go on meeting at their barriers, storing nothing
                    if (ok) ok = mbar_wait_bounded(tfull0 + 8 * slot, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    const int at = h ? w.at1 : 0, valid = min(h ? w.n1 : w.n0, w.ntok - at);
                    __nv_bfloat16 *dst = out + ((int64_t)w.row0 + at) * p.ldo + m + col;
#pragma unroll 1
                    for (int g = 0; g < valid; g += 32, buf ^= 1) {
                        uint32_t v[32];
                        tmem_ld32(lane_base + slot * 256 + g, v);
                        const uint32_t sb = smem_u32(stage) + buf * 8192u;
                        const uint32_t sw = sb + (uint32_t)(warp * 32 + lane) * 2u;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const __nv_bfloat16 x = __float2bfloat16_rn(__uint_as_float(v[i]));
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(sw + (uint32_t)i * 256u), "h"(*reinterpret_cast<const uint16_t *>(&x)) : "memory");
                        }
                        // one barrier per group: a buffer is written again after the next group's barrier,
                        // which every warp reaches after reading it
                        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = warp * 8 + q * 2 + (lane >> 4);
                            uint4 x;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                         : "r"(sb + (uint32_t)r * 256u + (uint32_t)col * 2u)
                                         : "memory");
                            if (ok && col_ok && g + r < valid) *reinterpret_cast<uint4 *>(dst + (int64_t)(g + r) * p.ldo) = x;
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(tempty_leader0 + 8 * slot);
                }
            }
            if (DIR == kExpWeight && !__all_sync(0xffffffffu, ok)) break;
        }
        if constexpr (DIR == kExpWeight) bulk_wait_all();
    }

    // no remote arrive or MMA may target a CTA that has left
    cluster_sync_all();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, 512);
    }
}

template <int DIR>
cudaError_t launch_dir(const ExpertPairParams &p, int grid, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_pair_kernel<DIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    experts_pair_kernel<DIR><<<grid, THREADS, SMEM, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_experts_pair(const ExpertPairParams &p, int dir, int grid, cudaStream_t s) {
    return dir == kExpForward ? launch_dir<kExpForward>(p, grid, s) : dir == kExpData ? launch_dir<kExpData>(p, grid, s) : launch_dir<kExpWeight>(p, grid, s);
}

}  // namespace cbd
