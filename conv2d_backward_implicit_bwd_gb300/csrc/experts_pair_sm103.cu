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
// A tile is 256 x up to 256 with two accumulators in TMEM, so the epilogue of
// one tile runs under the next one's MMAs.  (512 wide, single-buffered tiles
// move 48 KB instead of 64 KB per CTA for the same work, but their exposed
// epilogues cost more: 16384 x 1024 x 2048 forward 78 against 58 us, data
// 32768 x 2048 x 2048 217 against 189 us, weight 103 against 79 us.)
//
// Ragged ends.  Rows past an expert's end that a box brings along are other
// columns of D (forward, data), never stored.  For weight they would be
// summed: the partial block multiplies only its valid 16-row steps, and where the
// last step is partial a helper warp of each CTA zeroes its rows in shared
// memory after they have landed (both operands: 0 x NaN is NaN) before the MMA
// may read them.  That block is the first of its tile, so that the zeroing runs
// while the MMAs still work on the tile before (as the last one it cost 1.3 us a
// tile).
//
// Schedule.  Pair b of P takes tiles b, 2P - 1 - b, 2P + b, ... (back and forth,
// so that a fall or rise of the tiles' cost along the experts evens out).  One
// warp of each CTA builds the table and decodes the tiles ahead of the others.
// (Drawn from a counter by the leader, which hands them to both CTAs a tile ahead,
// they took 1% less; in falling cost order the sort took more than it gave.)
//
// Precision of weight.  The tensor core's accumulator truncates: over r rows the
// sum loses about r 2^-30 of itself (1.2e-6 measured at 1024 rows).  So weight
// starts a new accumulator every 512 rows and its epilogue adds those in fp32
// registers, which holds the error below 5e-7 for any number of rows; the add
// runs under the other accumulator's MMAs.
//
// Bounds, measured at 6.68 TB/s and 1963 TFLOP/s.  Tensor pipe: forward of 16384
// rows by 16 filters of 1024 x 2048 47 to 52 us (0.74 to 0.67 of the rate), data of
// 32768 rows by 32 of 2048 x 2048 163 (0.86, the rows of each expert uneven); called
// without a pause 54 and 191 under the power cap (1.6 and 1.4 GHz).  Memory: 256
// rows by 64 filters of 2048 x 1024 49 us (0.79; four rounds for 3.4 rounds' tiles);
// weight of the first of these, adding to fp32 gradients, 77 us (0.72; stored without
// adding 62).  Adding by reading the old gradient into the epilogue's staging and
// storing the sum was no faster (82 to 86 us against 78).
//
// Rows off the 16-byte lines (strides or addresses) cannot come by TMA.  Warps (eight;
// weight four, for both operands) read them in whole lines, shift them into place in
// registers and write the swizzled tile themselves; only lines inside the tensor are
// read whole.  The 16384 rows above with a stride of 1041: 98 us forward, 325 weight
// (on warp-level MMAs 511 and 547).  Bound by the way of a k-block through a warp, its
// shuffles and shifts: two in flight, in weight three batches of eight, with the
// registers that the sums leave.  Output rows off the lines leave in single elements:
// 66 us.
//
// Roles per CTA, in warps: epilogue 4 (weight 8, with most of the registers), A
// loads 1, MMA (leader CTA) and TMEM 1, B loads 2 (off the lines 8), helper 1 (weight:
// partial blocks; else rows of no expert), schedule 1.  Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <type_traits>

#include "device_util.cuh"
#include "expert_table.cuh"
#include "internal.h"
#include "lines.cuh"
#include "tc_common.cuh"
#include "tc_pair.cuh"
#include "train.h"

namespace cbd {

namespace {

constexpr int RING = 4;  // tiles between the schedule and its readers
constexpr int WIDE = 256;
constexpr int A_BYTES = 128 * 64 * 2;
constexpr int B_BYTES = 128 * 64 * 2;  // one CTA's half of the tile's columns
constexpr int SEGMENT = 8;             // weight: k-blocks (of 64 rows) of one accumulator
constexpr int MAX_STAGES = 6;

struct Bars {
    ExpertRing<RING> ring;
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];
    uint64_t tail[MAX_STAGES], peer[MAX_STAGES];  // weight: partial blocks landed in this CTA; peer's rows zeroed
                                                  // (off the lines, tail: this CTA's warps have written)
    uint64_t tfull[2], tempty[2];
    int32_t vote[8];  // forward, data: what each epilogue warp drew, two tiles in turn
    uint32_t tmem;
    int32_t abort;
};
template <int DIR, bool LOOSE>
struct Cfg {
    static constexpr bool W = DIR == kExpWeight;
    static constexpr int B_WARPS = !LOOSE ? 2 : W ? 4 : 8;  // (weight off the lines: of both operands)
    static constexpr int S = W ? 5 : 6;                  // pipeline stages
    static constexpr int OUT_BYTES = W ? 32768 : 16384;  // epilogue staging
    static constexpr int EPI = W ? 8 : 4;                // epilogue warps 0 .. EPI - 1
    static constexpr int LOAD_A = EPI, MMA = EPI + 1, HELP = EPI + 2, SCHED = EPI + 3, LOAD_B = EPI + 4;
    static constexpr int THREADS = W || LOOSE ? 512 : 320;  // weight: two warpgroups of epilogue, two of the others
    static constexpr int SMEM = 1024 + S * (A_BYTES + B_BYTES) + OUT_BYTES + (int)sizeof(ExpertTable) + 8 + (int)sizeof(Bars);
    static_assert(SMEM <= 232448, "shared memory of one CTA");
};

// (bar in this CTA)
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// What this CTA's threads have written to its shared memory, and a fence.proxy.async has made visible to the MMA, is ready:
// a release at cluster scope, as the other CTA's MMA warp waits for it, of shared memory alone.  (A release of everything
// waits for the loads that the SM has in flight: 16384 rows by 16 filters of 1024 x 2048 off the lines 130 us forward and
// 152 data instead of 110 and 117; from four warps in turn 144 and 155.)
__device__ __forceinline__ void arrive_written(uint32_t cluster_addr) {
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
        : "memory");
}
template <int DIR>
__device__ __forceinline__ ExpertWork decode(const ExpertPairParams &p, const ExpertTable &tab, int mt, int t) {
    ExpertWork w;
    w.e = expert_of_tile(tab, p.experts, t);
    const int l = t - tab.tile[w.e], len = tab.len(w.e), q = l / mt;
    w.m0 = (l - q * mt) * 256;
    w.kb0 = 0;
    if constexpr (DIR == kExpWeight) {
        w.row0 = tab.off[w.e];
        w.ntok = q * WIDE;  // first column
        w.kb1 = (len + 63) / 64;  // 0: an expert without rows
        w.last = len - (w.kb1 - 1) * 64;
        w.n = WIDE;
    } else {
        const int size = chunk_rows(len), first = q * size;
        w.row0 = tab.off[w.e] + first;
        w.ntok = min(size, len - first);
        w.n = (w.ntok + 31) & ~31;
        w.kb1 = ((DIR == kExpForward ? p.K : p.N) + 63) / 64;
        w.last = 64;  // past the depth both operands read as zero
    }
    return w;
}

template <int DIR, bool LOOSE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg<DIR, LOOSE>::THREADS, 1) experts_pair_kernel(const __grid_constant__ ExpertPairParams p) {
    using C = Cfg<DIR, LOOSE>;
    constexpr int S = C::S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sA = smem, *sB = smem + S * A_BYTES;
    uint8_t *stage = sB + S * B_BYTES;
    Bars &bars = *reinterpret_cast<Bars *>(stage + C::OUT_BYTES);
    ExpertTable &tab = *reinterpret_cast<ExpertTable *>(stage + C::OUT_BYTES + (sizeof(Bars) + 7) / 8 * 8);
    volatile int32_t *abort_flag = &bars.abort;

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tail0 = smem_u32(bars.tail),
                   peer0 = smem_u32(bars.peer), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int mdim = DIR == kExpData ? p.K : p.N;
    const int mt = (mdim + 255) / 256;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, (LOOSE && C::W ? 0 : 1) + (LOOSE ? 2 : 0));
            mbar_init(empty0 + 8 * s, 1);
            mbar_init(tail0 + 8 * s, LOOSE ? C::B_WARPS : 1);
            mbar_init(peer0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * C::EPI);  // epilogue warps of both CTAs
        }
        // B loads, epilogue, the leader's MMA; A loads (not in weight off the lines); the helper (weight, off the lines)
        bars.ring.init(C::B_WARPS + C::EPI + (leader ? 1 : 0) + (LOOSE && C::W ? 0 : 1) + (LOOSE || C::W ? 1 : 0));
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == C::MMA) {
        tmem_alloc2(smem_u32(&bars.tmem), 512);
        tc_fence_before();
    }
    if (warp == C::LOAD_A && lane == 0) {
        if (!(LOOSE && C::W)) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.a)) : "memory");
        if (!LOOSE) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.b)) : "memory");
    }
    cluster_sync_all();
    tc_fence_after();
    pdl_next();
    if (warp == C::SCHED)
        build_expert_table_early(tab, p.offsets, &bars.abort, p.experts, p.rows, DIR == kExpWeight ? kMaxRows : WIDE,
                                 DIR == kExpWeight ? mt * ((p.K + WIDE - 1) / WIDE) : mt, DIR == kExpWeight && !p.accumulate,
                                 blockIdx.x == 0 ? p.status : nullptr);
    else
        pdl_wait();
    const uint32_t tmem_base = bars.tmem;
    if (threadIdx.x == 0 && !leader) {
        // the pair's MMAs write this CTA's rows at the leader's TMEM address
        if (ld_shared_cluster_u32(mapa_shared(smem_u32(&bars.tmem), 0)) != tmem_base) record_status(p.status, kDevFaultIndex);
    }

    // weight: 128 registers a thread at launch (512 threads), 192 for the epilogue with its sums, 64 for the others (off
    // the lines 160 and 96)
    if (warp < C::EPI) {
        if constexpr (DIR == kExpWeight) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LOOSE ? 160 : 192));
        // ------------------------------------------------------------ epilogue (both CTAs)
        const uint32_t tempty_leader0 = mapa_shared(tempty0, 0);
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp % 4) * 32) << 16);
        uint32_t use = 0, buf = 0;
        bool ok = true;
        for (uint32_t i = 0;; ++i) {
            const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
            bool more = __all_sync(0xffffffffu, w.n != 0);
            if (more && lane == 0) bars.ring.done(i);
            if constexpr (DIR != kExpWeight) {
                // the four warps meet at barriers below: they go on or stop together
                volatile int32_t *vote = bars.vote + (i & 1) * 4;
                if (lane == 0) vote[warp] = more;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                more = vote[0] & vote[1] & vote[2] & vote[3];
            }
            if (!more) break;
            const int m = w.m0 + (int)rank * 128;
            if constexpr (DIR == kExpWeight) {
                // this warp's 32 rows x 128 columns, summed over the accumulators in registers
                constexpr int COLS = WIDE / 2;
                const int mrow = m + (warp % 4) * 32, col0 = (warp / 4) * COLS;
                float sum[COLS];
#pragma unroll
                for (int q = 0; q < COLS; ++q) sum[q] = 0.f;
                for (int left = w.kb1; left > 0; left -= SEGMENT, ++use) {
                    const uint32_t b = use & 1;
                    if (ok) ok = mbar_wait_bounded(tfull0 + 8 * b, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
#pragma unroll
                    for (int g = 0; g < COLS / 16; ++g) {
                        uint32_t v[16];
                        tmem_ld16(lane_base + b * 256 + col0 + g * 16, v);
#pragma unroll
                        for (int q = 0; q < 16; ++q) sum[g * 16 + q] += __uint_as_float(v[q]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_relaxed(tempty_leader0 + 8 * b);
                }
                // 32 x 32 pieces (128 bytes of a row) through swizzled staging and TMA stores, added in L2 when
                // accumulating: one writer per element, so the order is fixed
                uint8_t *slab = stage + warp * 4096;
#pragma unroll
                for (int g = 0; g < COLS / 32; ++g) {
                    const int col = w.ntok + col0 + g * 32;
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                    const uint32_t sb = smem_u32(slab) + (uint32_t)lane * 128u;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (((uint32_t)q ^ (lane & 7)) << 4)),
                                     "f"(sum[g * 32 + 4 * q]), "f"(sum[g * 32 + 4 * q + 1]), "f"(sum[g * 32 + 4 * q + 2]), "f"(sum[g * 32 + 4 * q + 3])
                                     : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (ok && lane == 0 && mrow < p.N && col < p.K) {
                        const uint64_t map = reinterpret_cast<uint64_t>(&p.o);
                        if (p.accumulate)
                            asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                                         "r"(col), "r"(mrow), "r"(w.e), "r"(smem_u32(slab))
                                         : "memory");
                        else
                            asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                                         "r"(col), "r"(mrow), "r"(w.e), "r"(smem_u32(slab))
                                         : "memory");
                        bulk_commit();
                    }
                }
            } else {
                const uint32_t b = use & 1, acc = lane_base + b * 256;
                // after a wait that ran out the warps go on meeting at their barriers, storing nothing
                if (ok) ok = mbar_wait_bounded(tfull0 + 8 * b, (use >> 1) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                ++use;
                // columns of the accumulator are rows of the output: 32 of them at a time are turned around in
                // shared memory ([row][128 of the M dimension], 256 bytes) and leave in 16-byte stores, two
                // whole row segments to an instruction.  (A bulk copy per row took 95 clocks each: 25 us for
                // 512 rows.)
                const int col = (lane & 15) * 8;
                const bool col_ok = m + col < mdim;
                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + (int64_t)w.row0 * p.ldo + m + col;
#pragma unroll 1
                for (int g = 0; g < w.ntok; g += 32, buf ^= 1) {
                    uint32_t v[32];
                    tmem_ld32(acc + g, v);
                    const uint32_t sb = smem_u32(stage) + buf * 8192u;
                    const uint32_t sw = sb + (uint32_t)(warp * 32 + lane) * 2u;
#pragma unroll
                    for (int q = 0; q < 32; ++q) {
                        const __nv_bfloat16 x = __float2bfloat16_rn(__uint_as_float(v[q]));
                        asm volatile("st.shared.b16 [%0], %1;" ::"r"(sw + (uint32_t)q * 256u), "h"(*reinterpret_cast<const uint16_t *>(&x)) : "memory");
                    }
                    // one barrier per group: a buffer is written again after the next group's barrier, which
                    // every warp reaches after reading it
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (!p.out_lines) {
                        // element by element, 32 neighbours an instruction
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            const int r = warp * 8 + q / 4, c = q % 4 * 32 + lane;
                            uint16_t x;
                            asm volatile("ld.shared.b16 %0, [%1];" : "=h"(x) : "r"(sb + (uint32_t)r * 256u + (uint32_t)c * 2u) : "memory");
                            if (ok && m + c < mdim && g + r < w.ntok) *reinterpret_cast<uint16_t *>(dst - col + c + (int64_t)(g + r) * p.ldo) = x;
                        }
                        continue;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int r = warp * 8 + q * 2 + (lane >> 4);
                        uint4 x;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"(sb + (uint32_t)r * 256u + (uint32_t)col * 2u)
                                     : "memory");
                        if (ok && col_ok && g + r < w.ntok) *reinterpret_cast<uint4 *>(dst + (int64_t)(g + r) * p.ldo) = x;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_relaxed(tempty_leader0 + 8 * b);
            }
        }
        if constexpr (DIR == kExpWeight) bulk_wait_all();
    } else {
        if constexpr (DIR == kExpWeight) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LOOSE ? 96 : 64));
        if (warp == C::SCHED) {
            // ------------------------------------------------------------ schedule
            if constexpr (DIR != kExpWeight) asm volatile("bar.arrive 2, 64;" ::: "memory");
            if (lane == 0) {
                const int total = tab.tile[p.experts];
                for (uint32_t i = 0;; ++i) {
                    const int t = (int)i * npairs + ((i & 1) ? npairs - 1 - pair : pair);
                    ExpertWork w;
                    w.n = 0;
                    // (the last round may be short: a pair beyond it has nothing there and nothing after)
                    if (t < total) w = decode<DIR>(p, tab, mt, t);
                    if (!bars.ring.give(i, w, p.wait_budget, abort_flag, p.status) || w.n == 0) break;
                }
            }
            __syncwarp();
        } else if (LOOSE && warp >= C::LOAD_B) {
            if constexpr (LOOSE && DIR == kExpWeight) {
                // -------------------------------------------------------- weight: rows that TMA cannot load, both operands
                // A k-block in eight batches of 16 rows, four of dy and four of x, three in flight.  A thread takes line
                // c of each half of a row's 256 bytes; what follows the second half's last is c = 0's third line.  Rows
                // past the expert's end are zeros.
                const int th = threadIdx.x - C::LOAD_B * 32, c = th & 7, r0 = th >> 3;
                const uint32_t to = (uint32_t)r0 * 128u + (uint32_t)((c ^ (r0 & 7)) << 4);
                const int from = (lane & 24) | ((lane + 1) & 7);
                struct Batch {
                    uint4 x0, x1, after;
                    int shift;
                };
                uint32_t it = 0;
                bool ok = true;
                for (uint32_t i = 0; ok; ++i) {
                    const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!__all_sync(0xffffffffu, w.n != 0)) break;
                    if (lane == 0) bars.ring.done(i);
                    // batch f of the tile: k-block f / 8 (the partial one first), rows 16 (f & 3) on, of dy if !(f & 4)
                    const int batches = w.kb1 * 8;
                    auto within = [&](const void *first, const void *last, int64_t ld, int col) {
                        const uintptr_t b = reinterpret_cast<uintptr_t>(first), head = b + (uintptr_t)(((int64_t)w.row0 * ld + col) * 2);
                        const uintptr_t tail = head + (uintptr_t)((int64_t)((w.kb1 - 1) * 64 + w.last - 1) * ld * 2);
                        return (head & ~uintptr_t(15)) >= b && (tail & ~uintptr_t(15)) + 272 <= reinterpret_cast<uintptr_t>(last);
                    };
                    const bool inside = within(p.rows_at, p.rows_end, p.ldb, w.m0 + (int)rank * 128) && within(p.rows2_at, p.rows2_end, p.ldb2, w.ntok + (int)rank * 128);
                    auto fetch = [&](auto whole, int f, Batch &x) {
                        const int kb = f >> 3, r = (f & 3) * 16 + r0, valid = kb == 0 ? w.last : 64;
                        x.x0 = x.x1 = x.after = make_uint4(0u, 0u, 0u, 0u);
                        x.shift = 0;
                        const bool there = f < batches && r < valid;
                        const bool b = f & 4;
                        const uintptr_t begin = reinterpret_cast<uintptr_t>(b ? p.rows2_at : p.rows_at), end = reinterpret_cast<uintptr_t>(b ? p.rows2_end : p.rows_end);
                        const int col = (b ? w.ntok : w.m0) + (int)rank * 128;
                        const int64_t row = (int64_t)w.row0 + (kb == 0 ? w.kb1 - 1 : kb - 1) * 64 + r;
                        const uintptr_t at = begin + (uintptr_t)((row * (b ? p.ldb2 : p.ldb) + col) * 2), line = (at & ~uintptr_t(15)) + 16 * c;
                        x.shift = (int)(at & 15) / 2;
                        if constexpr (decltype(whole)::value) {
                            if (there) {
                                x.x0 = *reinterpret_cast<const uint4 *>(line);
                                x.x1 = *reinterpret_cast<const uint4 *>(line + 128);
                            }
                            if (there && c == 0) x.after = *reinterpret_cast<const uint4 *>(line + 256);
                        } else if (there) {
                            x.x0 = load_line(line, begin, end);
                            x.x1 = load_line(line + 128, begin, end);
                            if (c == 0 && x.shift) x.after = load_line(line + 256, begin, end);
                        }
                    };
                    auto park = [&](int f, const Batch &x) {
                        const uint32_t s = it % S, ph = (it / S) & 1;
                        if ((f & 7) == 0) {
                            ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer));
                            if (!ok) return;
                        }
                        const uint4 a = c == 0 ? x.x1 : x.x0, b = c == 0 ? x.after : x.x1;
                        uint4 h0, h1;
                        h0.x = __shfl_sync(0xffffffffu, a.x, from);
                        h0.y = __shfl_sync(0xffffffffu, a.y, from);
                        h0.z = __shfl_sync(0xffffffffu, a.z, from);
                        h0.w = __shfl_sync(0xffffffffu, a.w, from);
                        h1.x = __shfl_sync(0xffffffffu, b.x, from);
                        h1.y = __shfl_sync(0xffffffffu, b.y, from);
                        h1.z = __shfl_sync(0xffffffffu, b.z, from);
                        h1.w = __shfl_sync(0xffffffffu, b.w, from);
                        const uint4 v0 = shifted(x.x0, h0, x.shift), v1 = shifted(x.x1, h1, x.shift);
                        const uint32_t dst = ((f & 4) ? smem_u32(sB + s * B_BYTES) : smem_u32(sA + s * A_BYTES)) + (uint32_t)(f & 3) * 2048u + to;
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v0.x), "r"(v0.y), "r"(v0.z), "r"(v0.w) : "memory");
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 8192u), "r"(v1.x), "r"(v1.y), "r"(v1.z), "r"(v1.w) : "memory");
                        if ((f & 7) == 7) {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(tail0 + 8 * s);
                            ++it;
                        }
                    };
                    auto run = [&](auto whole) {
                        Batch b0, b1, b2, b3;
                        fetch(whole, 0, b0);
                        fetch(whole, 1, b1);
                        fetch(whole, 2, b2);
#pragma unroll 1
                        for (int f = 0; f < batches && ok; f += 4) {
                            fetch(whole, f + 3, b3);
                            park(f, b0);
                            if (!ok) break;
                            fetch(whole, f + 4, b0);
                            park(f + 1, b1);
                            fetch(whole, f + 5, b1);
                            park(f + 2, b2);
                            fetch(whole, f + 6, b2);
                            park(f + 3, b3);
                        }
                    };
                    if (inside)
                        run(std::true_type());
                    else
                        run(std::false_type());
                }
            } else if constexpr (LOOSE) {
                // -------------------------------------------------------- rows that TMA cannot load
                // A thread takes line c of a row's 128 bytes of a k-block, of rows 32 apart, two k-blocks in flight; the
                // eight elements that belong together lie on its line and the next thread's (of the last, the next
                // k-block's first).  Shifted, they go where TMA would put them.  Rows past the tile are other columns of
                // D: they stay as they are.
                const int th = threadIdx.x - C::LOAD_B * 32, c = th & 7, r0 = th >> 3;
                const uint32_t to = (uint32_t)r0 * 128u + (uint32_t)((c ^ (r0 & 7)) << 4);
                const int depth = DIR == kExpForward ? p.K : p.N;
                const uintptr_t begin = reinterpret_cast<uintptr_t>(p.rows_at), end = reinterpret_cast<uintptr_t>(p.rows_end);
                uint32_t it = 0;
                bool ok = true;
                for (uint32_t i = 0; ok; ++i) {
                    const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!__all_sync(0xffffffffu, w.n != 0)) break;
                    if (lane == 0) bars.ring.done(i);
                    const int half = w.n / 2, at = (int)rank * half;
                    uintptr_t src[4];  // first line of the row, in its low bits the row's first element there
                    bool in[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = r0 + 32 * j;
                        in[j] = r < half && at + r < w.ntok;
                        src[j] = begin + (uintptr_t)((int64_t)(w.row0 + (in[j] ? at + r : 0)) * p.ldb * 2);
                    }
                    const bool any = __any_sync(0xffffffffu, in[0]), more = __any_sync(0xffffffffu, in[1]);
                    // all lines of the tile inside the tensor?  (else the loads would meet a branch each, and wait there)
                    const int rows_here = min(half, w.ntok - at);
                    const uintptr_t head = begin + (uintptr_t)((int64_t)(w.row0 + at) * p.ldb * 2), tail = head + (uintptr_t)((int64_t)(rows_here - 1) * p.ldb * 2) + 2 * (uintptr_t)depth;
                    const bool inside = (head & ~uintptr_t(15)) >= begin && ((tail + 15) & ~uintptr_t(15)) <= end;
                    auto fetch = [&](auto whole, int kb, uint4 (&x)[4]) {
                        const int off = kb * 128 + c * 16;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int s2 = (int)(src[j] & 15);
                            const uintptr_t line = src[j] - s2 + off;
                            x[j] = make_uint4(0u, 0u, 0u, 0u);
                            if (in[j] && off < depth * 2 + s2) {
                                if constexpr (decltype(whole)::value)
                                    x[j] = *reinterpret_cast<const uint4 *>(line);
                                else
                                    x[j] = load_line(line, begin, end);
                            }
                        }
                    };
                    auto park = [&](int kb, const uint4 (&x)[4], const uint4 (&next)[4]) {
                        const uint32_t s = it % S, ph = (it / S) & 1;
                        ++it;
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer));
                        if (!ok) return;
                        const uint32_t dst = smem_u32(sB + s * B_BYTES) + to;
                        const bool deep = kb * 64 + c * 8 < depth;  // (the depth is a multiple of 8)
                        const int from = (lane & 24) | ((lane + 1) & 7);
                        auto one = [&](int j) {
                            uint4 hi;
                            hi.x = __shfl_sync(0xffffffffu, c == 0 ? next[j].x : x[j].x, from);
                            hi.y = __shfl_sync(0xffffffffu, c == 0 ? next[j].y : x[j].y, from);
                            hi.z = __shfl_sync(0xffffffffu, c == 0 ? next[j].z : x[j].z, from);
                            hi.w = __shfl_sync(0xffffffffu, c == 0 ? next[j].w : x[j].w, from);
                            uint4 v = shifted(x[j], hi, (int)(src[j] & 15) / 2);
                            if (!deep) v = make_uint4(0u, 0u, 0u, 0u);
                            if (in[j])
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (uint32_t)j * 4096u), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                        };
                        // (a warp's four rows of j = 0 are the first to be there; without branches the four overlap)
                        if (more) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) one(j);
                        } else if (any) {
                            one(0);
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(tail0 + 8 * s);
                    };
                    auto run = [&](auto whole) {
                        uint4 x0[4], x1[4], x2[4], x3[4];
                        fetch(whole, 0, x0);
                        fetch(whole, 1, x1);
                        fetch(whole, 2, x2);
#pragma unroll 1
                        for (int kb = 0; kb < w.kb1 && ok; kb += 4) {
                            fetch(whole, kb + 3, x3);
                            park(kb, x0, x1);
                            if (kb + 1 >= w.kb1 || !ok) break;
                            fetch(whole, kb + 4, x0);
                            park(kb + 1, x1, x2);
                            if (kb + 2 >= w.kb1 || !ok) break;
                            fetch(whole, kb + 5, x1);
                            park(kb + 2, x2, x3);
                            if (kb + 3 >= w.kb1 || !ok) break;
                            fetch(whole, kb + 6, x2);
                            park(kb + 3, x3, x0);
                        }
                    };
                    if (inside || rows_here <= 0)
                        run(std::true_type());
                    else
                        run(std::false_type());
                }
            }
            __syncwarp();
        } else if (LOOSE && C::W && warp == C::LOAD_A) {
            // (the warps above load both operands)
        } else if (warp == C::LOAD_A || warp == C::LOAD_B || warp == C::LOAD_B + 1) {
            // ------------------------------------------------------------ loads
            if (lane == 0) {
                const uint32_t full_leader0 = mapa_shared(full0, 0);
                uint32_t it = 0;
                bool ok = true, issued = false;
                for (uint32_t i = 0; ok; ++i) {
                    const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (w.n == 0) break;
                    bars.ring.done(i);
                    // B columns of this CTA in boxes of 64, one for each B warp
                    const int half = w.n / 2, boxes = (half + 63) / 64, q = warp - C::LOAD_B;
                    const uint32_t bytes = (uint32_t)A_BYTES + 8192u * (uint32_t)boxes;  // of one CTA
                    const int at = (int)rank * half + 64 * q;
                    for (int kb = 0; kb < w.kb1; ++kb, ++it) {
                        const uint32_t s = it % S, ph = (it / S) & 1;
                        if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        // weight: the partial block first, with a partial last step through the helper warp, on
                        // this CTA's own barrier
                        const bool fix = DIR == kExpWeight && kb == 0 && (w.last & 15) != 0;
                        const int row = w.row0 + (kb == 0 ? w.kb1 - 1 : kb - 1) * 64;  // (weight)
                        const uint32_t bar = fix ? tail0 + 8 * s : full_leader0 + 8 * s;
                        if (warp == C::LOAD_A) {
                            if (fix)
                                mbar_arrive_expect_tx(tail0 + 8 * s, bytes);
                            else if (leader)
                                mbar_arrive_expect_tx(full0 + 8 * s, LOOSE ? 2u * A_BYTES : 2 * bytes);
                            const uint32_t dst = smem_u32(sA + s * A_BYTES);
                            const int m = w.m0 + (int)rank * 128;
                            if constexpr (DIR == kExpForward) {
                                tma_load_3d_pair(dst, &p.a, bar, kb * 64, m, w.e);
                            } else if constexpr (DIR == kExpData) {
                                tma_load_3d_pair(dst, &p.a, bar, m, kb * 64, w.e);
                                tma_load_3d_pair(dst + 8192, &p.a, bar, m + 64, kb * 64, w.e);
                            } else {
                                for (int b = 0; b < 2; ++b)
                                    if (fix)
                                        tma_load_2d(dst + 8192 * b, &p.a, bar, m + 64 * b, row);
                                    else
                                        tma_load_2d_pair(dst + 8192 * b, &p.a, bar, m + 64 * b, row);
                            }
                            issued = true;
                        } else if (q < boxes) {
                            const uint32_t dst = smem_u32(sB + s * B_BYTES + 8192 * q);
                            if constexpr (DIR == kExpWeight) {
                                if (fix)
                                    tma_load_2d(dst, &p.b, bar, w.ntok + at, row);
                                else
                                    tma_load_2d_pair(dst, &p.b, bar, w.ntok + at, row);
                            } else {
                                tma_load_2d_pair(dst, &p.b, bar, kb * 64, w.row0 + at);
                            }
                            issued = true;
                        }
                    }
                }
                if (!ok && issued) {
                    for (int q = 0; q < 100; ++q) __nanosleep(1000);
                }
            }
            __syncwarp();
        } else if (warp == C::MMA) {
            // ------------------------------------------------------------ MMA (leader)
            if (leader) {
                constexpr bool A_K = DIR == kExpForward, B_K = DIR != kExpWeight;
                constexpr uint32_t A_STEP = A_K ? 2 : 128, B_STEP = B_K ? 2 : 128;  // a 16-deep step, in 16 bytes
                const uint32_t idesc0 = (1u << 4) | (1u << 7) | (1u << 10) | ((A_K ? 0u : 1u) << 15) | ((B_K ? 0u : 1u) << 16) | ((uint32_t)(256 >> 4) << 24);
                const uint64_t a_desc0 = smem_desc_sw128(smem_u32(sA), A_K ? 16 : 8192, 1024);
                const uint64_t b_desc0 = smem_desc_sw128(smem_u32(sB), B_K ? 16 : 8192, 1024);
                const uint32_t a_lo = (uint32_t)a_desc0, a_hi = (uint32_t)(a_desc0 >> 32), b_lo = (uint32_t)b_desc0, b_hi = (uint32_t)(b_desc0 >> 32);
                uint32_t s = 0, ph = 0, use = 0;  // stage and its phase, accumulators used so far
                bool ok = true, issued = false;
                for (uint32_t i = 0; ok; ++i) {
                    ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutMma);
                    w.n = __shfl_sync(0xffffffffu, w.n, 0);
                    w.kb1 = __shfl_sync(0xffffffffu, w.kb1, 0);
                    w.last = __shfl_sync(0xffffffffu, w.last, 0);
                    if (w.n == 0) break;
                    if (lane == 0) bars.ring.done(i);
                    if (w.kb1 == 0) continue;
                    const uint32_t id = idesc0 | ((uint32_t)(w.n >> 3) << 17);
                    for (int left = w.kb1; left > 0 && ok;) {
                        // one accumulator: the whole depth, or a segment of it (weight)
                        const uint32_t b = use & 1, bph = (use >> 1) & 1, d = tmem_base + b * 256;
                        ++use;
                        // (both CTAs' epilogues arrive)
                        ok = __all_sync(0xffffffffu, wait_cluster(tempty0 + 8 * b, bph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                        if (!ok) break;
                        tc_fence_after();
                        uint32_t acc = 0;
                        const int end = DIR == kExpWeight && left > SEGMENT ? left - SEGMENT : 0;
                        for (; left > end; --left) {
                            // (LOOSE: the other CTA's warps wrote their half themselves)
                            const bool full = LOOSE ? wait_cluster(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma)
                                                    : mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma);
                            ok = __all_sync(0xffffffffu, full);
                            if (!ok) break;
                            const uint32_t ad = a_lo + s * (A_BYTES >> 4), bd = b_lo + s * (B_BYTES >> 4);
                            const int n = DIR == kExpWeight && left == w.kb1 ? (w.last + 15) / 16 : 4;
    #pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                if (kk < n) mma_pair_elect(d, ad + A_STEP * kk, a_hi, bd + B_STEP * kk, b_hi, id, acc);
                                acc = 1;
                            }
                            issued = true;
                            commit_pair_elect(empty0 + 8 * s);
                            if (++s == (uint32_t)S) {
                                s = 0;
                                ph ^= 1;
                            }
                        }
                        if (ok) commit_pair_elect(tfull0 + 8 * b);
                    }
                }
                if (!ok && issued) {
                    for (int q = 0; q < 100; ++q) __nanosleep(1000);
                }
            }
            __syncwarp();
        } else if (warp == C::HELP) {
            // ------------------------------------------------------------ helper: rows past an expert's end, rows of none
            if constexpr (LOOSE) {
                // What the load warps have written is made visible to the MMA from here: their own fence would wait for
                // the loads that they have in flight.
                if (lane == 0) {
                    const uint32_t full_leader0 = mapa_shared(full0, 0);
                    uint32_t it = 0;
                    bool ok = true;
                    for (uint32_t i = 0; ok; ++i) {
                        const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                        if (w.n == 0) break;
                        bars.ring.done(i);
                        for (int kb = 0; kb < w.kb1 && ok; ++kb, ++it) {
                            const uint32_t s = it % S, ph = (it / S) & 1;
                            ok = mbar_wait_bounded(tail0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                            if (!ok) break;
                            fence_proxy_async_smem();
                            arrive_written(full_leader0 + 8 * s);
                        }
                    }
                }
                __syncwarp();
            }
            if constexpr (DIR == kExpWeight && !LOOSE) {
                uint32_t it = 0, phase = 0;  // bit s: parity of the next use of tail[s] and peer[s]
                for (uint32_t i = 0;; ++i) {
                    const ExpertWork w = bars.ring.take(i, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!__all_sync(0xffffffffu, w.n != 0)) break;
                    if (lane == 0) bars.ring.done(i);
                    const uint32_t s = it % S, ph = (phase >> s) & 1;
                    it += (uint32_t)w.kb1;
                    if (w.kb1 == 0 || (w.last & 15) == 0) continue;
                    phase ^= 1u << s;
                    bool ok = mbar_wait_bounded(tail0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    // rows [last, next multiple of 16) of each 64 x 64 block: whole 128-byte lines, so the swizzle
                    // within a line does not matter
                    const int lo = w.last, n = ((lo + 15) & ~15) - lo;
                    uint8_t *line = sA + s * A_BYTES + lo * 128 + lane * 16;
                    uint8_t *line_b = sB + s * B_BYTES + lo * 128 + lane * 16;
                    for (int j = lane; j < n * 8; j += 32, line += 512, line_b += 512) {
                        *reinterpret_cast<uint4 *>(line) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(line + 8192) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(line_b) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(line_b + 8192) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (!leader) {
                            mbar_arrive_remote(mapa_shared(peer0 + 8 * s, 0));
                        } else {
                            ok = wait_cluster(peer0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                            if (ok) mbar_arrive(full0 + 8 * s);
                        }
                    }
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
            }
            if constexpr (DIR != kExpWeight) {
                // forward, data: rows of no expert get zeros (16-byte stores; the width is a multiple of 8)
                asm volatile("bar.sync 2, 64;" ::: "memory");  // the table
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
                const int lo = tab.off[0], hi = tab.off[p.experts], vec = mdim / 8;
                const int64_t nfill = (int64_t)lo + (p.rows - hi);
                for (int64_t f = blockIdx.x; f < nfill; f += gridDim.x) {
                    __nv_bfloat16 *at = out + (f < lo ? f : hi + (f - lo)) * p.ldo;
                    if (!p.out_lines) {
                        for (int c = lane; c < mdim; c += 32) at[c] = __nv_bfloat16(0.f);
                        continue;
                    }
                    uint4 *row = reinterpret_cast<uint4 *>(at);
                    for (int c = lane; c < vec; c += 32) row[c] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }

    // no remote arrive or MMA may target a CTA that has left
    cluster_sync_all();
    if (warp == C::MMA) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, 512);
    }
}

template <int DIR, bool LOOSE>
cudaError_t launch_dir(const ExpertPairParams &p, int grid, cudaStream_t s) {
    using C = Cfg<DIR, LOOSE>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(experts_pair_kernel<DIR, LOOSE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(experts_pair_kernel<DIR, LOOSE>, grid, C::THREADS, C::SMEM, s, p);
}

}  // namespace

cudaError_t launch_experts_pair(const ExpertPairParams &p, int dir, int grid, cudaStream_t s) {
    if (p.rows_at)
        return dir == kExpForward ? launch_dir<kExpForward, true>(p, grid, s) : dir == kExpData ? launch_dir<kExpData, true>(p, grid, s) : launch_dir<kExpWeight, true>(p, grid, s);
    return dir == kExpForward ? launch_dir<kExpForward, false>(p, grid, s) : dir == kExpData ? launch_dir<kExpData, false>(p, grid, s) : launch_dir<kExpWeight, false>(p, grid, s);
}

}  // namespace cbd
