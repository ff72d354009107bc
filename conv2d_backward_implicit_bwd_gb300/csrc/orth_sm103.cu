// orth_sm103.cu -- Newton-Schulz orthogonalisation of matrices: X <- a X + b (X X^T) X + c (X X^T)^2 X, `steps` times, from
// X = u / |u|_F.
//
// With the smaller side as the Gram side (X^T X for high matrices, from the right):
//   gram     A = X X^T                  or X^T X
//   square   B = c A A + b A + a I
//   product  X' = B X                   or X B
// three products a step; where X is large beside A, up to three steps go together: all is polynomials of A, which commute, so
//   T = B A, A' = T B, B' = c A' A' + b A' + a I, Q = B' B (, T' = B' A', A'' = T' B', B'' = ..., Q' = B'' Q)
//   X' = Q X                 or X Q
// with two products over the larger side where there were four (six), and symmetric ones instead.  (1024 x 2048, five steps
// in fp32: the error of three and two joined is that of steps apart on spectra flat, falling and of few directions over
// noise; all five joined lose ten times as much beside small singular values.)
//
// The products of polynomials are symmetric: of their results only the blocks of 256 from the diagonal on are
// computed and kept, and where an operand lies below it the block above is read across.  (Written transposed as well, each
// tile took 2 to 5 us longer.)
//
// Schedule.  One cooperative launch does all the products: a list of tiles in order of product, then matrix; pair b of P
// takes tiles b, b + P, ...  A tile begins when its matrix's tiles of the products before are done (a counter for each
// matrix), which in a batch is long past when the list comes round: no product ends with idle SMs, and there is one launch
// instead of fifteen.  (The tile with the lowest number that is not done waits for none that is not, and its pair is at it: the
// waits end.)  Where a product has fewer tiles than there are pairs its contraction is split, and the warp that comes last
// adds the pieces' sums in order.
//
// Precision.  A small singular value grows by a = 3.44 a step, and with it what a rounding has put beside it: one fp16
// or bf16 product each leaves 0.4 to 4 % (simulated on matrices of falling spectrum), above what a bf16 result holds.
// So the matrices between the products are pairs of fp16, hi + lo (22 bits), times 2^10 (the polynomial B 2^8) so that lo
// stays a normal number; a product is hi hi + hi lo + lo hi, on the tensor cores in fp32.  (fp16 rather than bf16: 22 bits
// instead of 16 at the same rate.  Singular values stay below 1.3 with the usual coefficients; B may reach 255, which the
// host's bound of 32 on each coefficient keeps below singular values of 1.5; what is joined the host has followed.)  The
// accumulator truncates, about 2^-26 of the sum with each instruction; a new one is begun every `segment` k-blocks and
// added in fp32 registers, under the other accumulator's MMAs.  Every two k-blocks the result's error is that of the same
// products in fp32 (8 directions over 1 % noise, 1024 x 1024: 4.6e-5, in fp32 4.5e-5; every eight 1.4e-4), but the sums take
// power, and power is what bounds large batches: 32 of 1024 x 2048 2226 us every eight, 2443 every two.  So plans of fp32 take two, and
// those of bf16, whose inputs were rounded by 1.7e-3 of their norm, eight.  (A last product of the hi halves alone would be 5 to 7 % of
// the time less, 32 of 1024 x 2048 2101 instead of 2226 us, but a bf16 result would be off by more than its own rounding:
// by 1.3e-3 of its norm from the rounded exact one, like this by 2e-4.)
//
// The tile is 256 x W on a pair of SMs (tcgen05 cta_group::2), two accumulators in TMEM; a k-block of 64 brings both
// halves of both operands, 64 KB a CTA for W = 256, and feeds twelve 16-deep MMAs, so loads are a third of what a plain
// product of the same rate would need.
//
// Roles per CTA, in warps: epilogue 8 (with most of the registers for the sums), A loads 1, B loads 1, MMA (leader CTA) and
// TMEM 1.  Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "device_util.cuh"
#include "internal.h"
#include "rows_io.cuh"
#include "tc_common.cuh"
#include "tc_pair.cuh"
#include "train.h"

namespace cbd {

namespace {

constexpr int EPI = 8, LOAD_A = 8, LOAD_B = 9, MMA = 10, THREADS = 512;
constexpr int A_BYTES = 128 * 64 * 2;  // of one plane of a stage
constexpr int OUT_BYTES = EPI * 4096;
constexpr int MOST_STAGES = 4;
constexpr int READY = 8;  // more than the pieces that the A loads can be ahead of the epilogue (a piece fills a stage at least)
static_assert(READY > MOST_STAGES + 2, "a barrier is not used again before everyone has seen it");

template <int W>
struct Cfg {
    static constexpr int B_BYTES = W / 2 * 64 * 2;  // one CTA's half of the tile's columns
    static constexpr int STAGE = 2 * (A_BYTES + B_BYTES);
    static constexpr int S = W == 256 ? 3 : 4;
};
struct Bars {
    uint64_t full[MOST_STAGES], empty[MOST_STAGES], tfull[2], tempty[2];
    uint64_t ready[READY];  // the operands of a piece are there, pieces in turn
    uint64_t old[EPI];      // a warp's part of A has come
    uint32_t tmem;
    int32_t abort;
};
template <int W>
constexpr int smem_bytes() {
    return 1024 + Cfg<W>::S * Cfg<W>::STAGE + OUT_BYTES + (int)sizeof(Bars);
}
static_assert(smem_bytes<256>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory of one CTA");

// One piece of the work: matrix e's tile in a phase, the contraction's blocks [kb0, kb1).
struct Work {
    int kind, a, b, e, tile, split;
    int m0, n0, n;  // first row and column, columns (a multiple of 32)
    int kb0, kb1;
    int M, N;
    bool poly, last;
};
// The i-th piece; ph: the phase of an earlier one.
template <int W>
__device__ __forceinline__ Work work_at(const OrthParams &p, int i, int &ph) {
    Work w;
    while (i >= p.phase[ph + 1].first) ++ph;
    const OrthPhase &f = p.phase[ph];
    i -= f.first;
    w.kind = f.kind;
    w.a = f.a;
    w.b = f.b;
    w.poly = f.poly;
    w.last = f.last;
    const int tiles = w.kind == kOrthProduct ? p.tiles_all : p.tiles_sym, splits = p.splits[w.kind];
    w.e = i / (tiles * splits);
    i -= w.e * tiles * splits;
    w.tile = i / splits;
    w.split = i - w.tile * splits;
    const int g = min(p.rows, p.cols);
    w.M = w.kind == kOrthProduct ? p.rows : g;
    w.N = w.kind == kOrthProduct ? p.cols : g;
    const int nt = (w.N + W - 1) / W;
    int l = w.tile, tm, tn;
    if (w.kind != kOrthProduct) {  // from the diagonal block on
        tm = 0;
        for (int len = nt; l >= len; len -= 256 / W) {
            l -= len;
            ++tm;
        }
        tn = tm * (256 / W) + l;
    } else {
        tm = l / nt;
        tn = l - tm * nt;
    }
    w.m0 = tm * 256;
    w.n0 = tn * W;
    w.n = min(W, (w.N - w.n0 + 31) & ~31);
    const int kblocks = ((w.kind == kOrthGram ? max(p.rows, p.cols) : g) + 63) / 64;
    w.kb0 = (int)((int64_t)kblocks * w.split / splits);
    w.kb1 = (int)((int64_t)kblocks * (w.split + 1) / splits);
    return w;
}
// Whether an operand's lines run across the contraction in its k-block kb: X's in X^T X, and where it is multiplied from the
// left; those of the symmetric matrices, of which only the blocks of 256 from the diagonal on are there, below it.
__device__ __forceinline__ bool a_across(const Work &w, bool high, int kb) { return w.a > 1 ? (kb >> 2) < (w.m0 >> 8) : w.kind == kOrthGram && high; }
__device__ __forceinline__ bool b_across(const Work &w, bool high, int kb) { return w.b > 1 ? (kb >> 2) < (w.n0 >> 8) : w.kind == kOrthProduct || high; }
__device__ __forceinline__ bool wait_done(const OrthParams &p, const Work &w, int want, volatile int32_t *abort, int32_t code) {
    const int32_t *at = p.done + w.e;
    if (ld_acquire_gpu(at) >= want) return true;
    const long long t0 = clock64();
    for (uint32_t it = 1;; ++it) {
        if (ld_acquire_gpu(at) >= want) return true;
        if ((it & 63) == 0) {
            if (*abort) return false;
            if (clock64() - t0 > p.wait_budget) {
                record_status(p.status, code);
                *abort = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ uint32_t pack_hi(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_lo(float x, float y) {
    const float2 h = __half22float2(__floats2half2_rn(x, y));
    return pack_hi(x - h.x, y - h.y);
}
__device__ __forceinline__ void store_box(const CUtensorMap *map, uint32_t src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
    bulk_commit();
}

__device__ __forceinline__ void load_box(const CUtensorMap *map, uint32_t dst, uint32_t bar, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

// One warp's 32 rows x COLS columns of a tile, in registers, to the planes hi and lo.
template <int COLS>
__device__ __forceinline__ void store_planes(const CUtensorMap *out, const Work &w, const float (&v)[COLS], uint8_t *slab, int row, int col, int lane) {
    const uint32_t sb = smem_u32(slab);
#pragma unroll
    for (int g = 0; g < COLS / 64; ++g)
#pragma unroll
        for (int plane = 0; plane < 2; ++plane) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = v[g * 64 + q * 8 + 2 * i], y = v[g * 64 + q * 8 + 2 * i + 1];
                    u[i] = plane ? pack_lo(x, y) : pack_hi(x, y);
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (uint32_t)lane * 128u + (((uint32_t)q ^ (lane & 7)) << 4)), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row < w.M && col + g * 64 < w.N) store_box(out + plane, sb, col + g * 64, row, w.e);
        }
}

// The same to the caller's tensors: the result itself, or the step on the weights.
template <int COLS>
__device__ __forceinline__ void store_result(const OrthParams &p, const Work &w, const float (&v)[COLS], uint8_t *slab, int row, int col, int lane) {
    const uint32_t sb = smem_u32(slab);
#pragma unroll
    for (int g = 0; g < COLS / 32; ++g) {
        if (lane == 0) bulk_wait_read();  // (of the product before)
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (uint32_t)lane * 128u + (((uint32_t)q ^ (lane & 7)) << 4)),
                         "f"(v[g * 32 + 4 * q]), "f"(v[g * 32 + 4 * q + 1]), "f"(v[g * 32 + 4 * q + 2]), "f"(v[g * 32 + 4 * q + 3])
                         : "memory");
        __syncwarp();
        const int c = col + g * 32 + lane;
        if (c >= w.N) continue;
        for (int r0 = 0; r0 < 32 && row + r0 < w.M; r0 += 8) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i]) : "r"(sb + (uint32_t)r * 128u + (((uint32_t)(lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4u) : "memory");
            }
            const int64_t at = (int64_t)w.e * p.lse + (int64_t)(row + r0) * p.ldo + c;
            if (p.weight) {
                float old[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) old[i] = row + r0 + i < w.M ? p.weight[at + i * p.ldo] : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (row + r0 + i >= w.M) break;
                    const float n = fmaf(-p.rate, x[i], old[i] * p.keep);
                    p.weight[at + i * p.ldo] = n;
                    if (p.copy) p.copy[at + i * p.ldo] = __float2bfloat16_rn(n);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (row + r0 + i >= w.M) break;
                    if (p.bf16)
                        static_cast<__nv_bfloat16 *>(p.result)[at + i * p.ldo] = __float2bfloat16_rn(x[i]);
                    else
                        static_cast<float *>(p.result)[at + i * p.ldo] = x[i];
                }
            }
        }
    }
}

// A tile whose contraction is split: every piece leaves its sums in the workspace, the warp that comes last adds them in
// order and goes on with the tile; false for the others.
template <int COLS>
__device__ __forceinline__ bool join_splits(const OrthParams &p, const Work &w, float (&sum)[COLS], int splits, int slice, int lane) {
    constexpr int STEP = 2 * EPI * 32 * COLS / 4;
    float4 *first = p.parts + (int64_t)orth_piece_place(p, w.e, w.tile, splits) * STEP + slice * (32 * COLS / 4) + lane;
#pragma unroll
    for (int q = 0; q < COLS / 4; ++q) __stcg(first + w.split * STEP + q * 32, make_float4(sum[4 * q], sum[4 * q + 1], sum[4 * q + 2], sum[4 * q + 3]));
    __syncwarp();
    int32_t *counter = p.arrived + orth_counter_place(p, w.e, w.tile) * 2 * EPI + slice;
    int before = 0;
    if (lane == 0) asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    before = __shfl_sync(0xffffffffu, before, 0);
    if (before != splits - 1) return false;
    if (lane == 0) *counter = 0;
    // 32 columns of the other pieces at once, so that one latency covers them
#pragma unroll
    for (int g = 0; g < COLS / 32; ++g) {
        float4 x[kOrthSplits - 1][8];
#pragma unroll
        for (int k = 0; k < kOrthSplits - 1; ++k) {
            const int from = k + (k >= w.split);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[k][q] = from < splits ? __ldcg(first + from * STEP + (g * 8 + q) * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int at = g * 32 + 4 * q;
            // ((piece 0 + piece 1) + piece 2): the sum of the first two does not depend on their order
            const float4 a = x[0][q], b = kOrthSplits > 2 ? x[kOrthSplits - 2][q] : make_float4(0.f, 0.f, 0.f, 0.f);
            static_assert(kOrthSplits == 3, "order of the pieces");
            auto in_order = [&](float own, float p, float r) { return w.split < 2 ? (own + p) + r : (p + r) + own; };
            sum[at] = in_order(sum[at], a.x, b.x);
            sum[at + 1] = in_order(sum[at + 1], a.y, b.y);
            sum[at + 2] = in_order(sum[at + 2], a.z, b.z);
            sum[at + 3] = in_order(sum[at + 3], a.w, b.w);
        }
    }
    return true;
}

template <int W>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) orth_kernel(const __grid_constant__ OrthParams p) {
    using C = Cfg<W>;
    constexpr int S = C::S, COLS = W / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stage = smem + S * C::STAGE;
    Bars &bars = *reinterpret_cast<Bars *>(stage + OUT_BYTES);
    volatile int32_t *abort_flag = &bars.abort;

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0, high = p.rows > p.cols;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty), ready0 = smem_u32(bars.ready);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2, total = p.phase[p.phases].first;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * EPI);  // epilogue warps of both CTAs
        }
        for (int i = 0; i < READY; ++i) mbar_init(ready0 + 8 * i, 1);
        for (int i = 0; i < EPI; ++i) mbar_init(smem_u32(&bars.old[i]), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == MMA) {
        tmem_alloc2(smem_u32(&bars.tmem), 512);
        tc_fence_before();
    }
    if (warp == LOAD_A) {  // the maps of the matrices that there are stand together
        const CUtensorMap *m = &p.maps[0].rows128[0];
        for (int i = lane; i < p.matrices * 6; i += 32) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m + i)) : "memory");
        __syncwarp();
    }
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = bars.tmem;
    if (threadIdx.x == 0 && !leader) {
        // the pair's MMAs write this CTA's rows at the leader's TMEM address
        if (ld_shared_cluster_u32(mapa_shared(smem_u32(&bars.tmem), 0)) != tmem_base) record_status(p.status, kDevFaultIndex);
    }

    // 128 registers a thread at launch (512 threads): 192 for the epilogue with its sums, 64 for the others
    if (warp < EPI) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // ------------------------------------------------------------ epilogue (both CTAs)
        const uint32_t tempty_leader0 = mapa_shared(tempty0, 0);
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp % 4) * 32) << 16);
        uint8_t *slab = stage + warp * 4096;
        uint32_t use = 0, piece = 0;
        int ph = 0;
        bool ok = true, fetching = false;
        const uint32_t old_bar = smem_u32(&bars.old[warp]);
        for (int i = pair; i < total; i += npairs, ++piece) {
            const Work w = work_at<W>(p, i, ph);
            const OrthPhase &f = p.phase[ph];
            const int row = w.m0 + (int)rank * 128 + (warp % 4) * 32, col0 = (warp / 4) * COLS, col = w.n0 + col0;
            // A polynomial adds to A, by other SMs in this launch.  Narrow tiles fetch their part under the MMAs, plane by plane
            // through the box that their results leave by; the hi half then waits in registers.  (Read from global memory, 16
            // bytes of a row to a lane, it held up the operands' loads: 300 x 300 137 us.)  Wide tiles, whose sums leave no
            // registers, read it past L1 afterwards, under the next tile's MMAs.
            constexpr bool AHEAD = W != 256;
            uint4 old_hi[AHEAD ? COLS / 8 : 1];
            auto fetch_old = [&](int plane) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_wait_read();
                    mbar_arrive_expect_tx(old_bar, 4096);
                    load_box(p.maps[w.a].store + plane, smem_u32(slab), old_bar, col, row, w.e);
                }
                __syncwarp();
            };
            auto wait_old = [&](int plane) {
                if (ok) ok = mbar_wait_bounded(old_bar, plane, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                ok = __all_sync(0xffffffffu, ok);
            };
            auto from_slab = [&](int q) { return *reinterpret_cast<const uint4 *>(slab + lane * 128 + ((q ^ (lane & 7)) << 4)); };
            auto from_memory = [&](int plane, int q) {
                const int r = row + lane, c = col + q * 8;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < w.M && c < p.pitch_gram) v = __ldcg(reinterpret_cast<const uint4 *>(p.at[w.a][plane] + ((int64_t)w.e * w.M + r) * p.pitch_gram + c));
                return v;
            };
            if (w.poly) {
                if (ok) ok = mbar_wait_bounded(ready0 + 8 * (piece % READY), (piece / READY) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                ok = __all_sync(0xffffffffu, ok);
                if constexpr (AHEAD) {
                    static_assert(W == 256 || COLS == 64, "a box for each plane");
                    if (ok) {
                        fence_proxy_async_global();
                        fetch_old(0);
                        fetching = true;
                        wait_old(0);
#pragma unroll
                        for (int q = 0; q < COLS / 8; ++q) old_hi[q] = from_slab(q);
                        if (ok) fetch_old(1);
                    }
                }
            }
            float sum[COLS];
#pragma unroll
            for (int q = 0; q < COLS; ++q) sum[q] = 0.f;
            for (int left = w.kb1 - w.kb0; left > 0; left -= p.segment, ++use) {
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
            if (AHEAD && w.poly) wait_old(1);
            if (!ok) continue;
            const int splits = p.splits[w.kind];
            if (W != 256 && splits > 1 && !join_splits<COLS>(p, w, sum, splits, (int)rank * EPI + warp, lane)) continue;
            if (w.poly) {
                // c sum + b A + a on the diagonal
                const float a = f.diag, b = f.add, c = f.mul;
                const int r = row + lane;
#pragma unroll
                for (int q = 0; q < COLS / 8; ++q) {
                    const uint4 h = AHEAD ? old_hi[AHEAD ? q : 0] : from_memory(0, q), l = AHEAD ? from_slab(q) : from_memory(1, q);
                    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&hw[k])), y = __half22float2(*reinterpret_cast<const __half2 *>(&lw[k]));
                        float &s0 = sum[q * 8 + 2 * k], &s1 = sum[q * 8 + 2 * k + 1];
                        s0 = fmaf(c, s0, b * (x.x + y.x));
                        s1 = fmaf(c, s1, b * (x.y + y.y));
                    }
                }
                if (col < row + 32 && row < col + COLS) {  // the diagonal's warps
#pragma unroll
                    for (int q = 0; q < COLS; ++q) sum[q] += r == col + q ? a : 0.f;
                }
            } else {
                const float mul = f.mul;
#pragma unroll
                for (int q = 0; q < COLS; ++q) sum[q] *= mul;
            }
            if (w.last) {
                store_result<COLS>(p, w, sum, slab, row, col, lane);
                continue;
            }
            store_planes<COLS>(p.maps[f.out].store, w, sum, slab, row, col, lane);
            // written, and known to be
            if (lane == 0) {
                bulk_wait_all();
                fence_proxy_async_global();
                asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p.done + w.e) : "memory");
            }
            __syncwarp();
        }
        if (!ok && fetching) {
            for (int q = 0; q < 100; ++q) __nanosleep(1000);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == LOAD_A || warp == LOAD_B) {
            // ------------------------------------------------------------ loads
            if (lane == 0) {
                const uint32_t full_leader0 = mapa_shared(full0, 0);
                uint32_t it = 0, piece = 0;
                int phase = 0;
                bool ok = true, issued = false;
                for (int i = pair; i < total && ok; i += npairs, ++piece) {
                    const Work w = work_at<W>(p, i, phase);
                    const int m = w.m0 + (int)rank * 128, n = w.n0 + (int)rank * (w.n / 2);
                    // What other SMs have written in this launch.  (One thread of a CTA asks for it: with every lane of the
                    // epilogue asking too, loads and counters took 3 us longer.)
                    const uint32_t bar_ready = ready0 + 8 * (piece % READY);
                    ok = warp == LOAD_A ? wait_done(p, w, p.phase[phase].need, abort_flag, kDevTimeoutProducer)
                                        : mbar_wait_bounded(bar_ready, (piece / READY) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!ok) break;
                    if (warp == LOAD_A) mbar_arrive(bar_ready);
                    fence_proxy_async_global();
                    // by lines along the contraction (this CTA's half of the tile in one box), and across it (in boxes of 64 x 64)
                    const OrthMaps &maps = p.maps[warp == LOAD_A ? w.a : w.b];
                    const CUtensorMap *along = warp == LOAD_A || W == 256 ? maps.rows128 : maps.rows64, *cross = maps.rows64;
                    for (int kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                        const uint32_t s = it % S, ph = (it / S) & 1;
                        if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = full_leader0 + 8 * s, to = smem_u32(smem + s * C::STAGE);
                        if (warp == LOAD_A && leader) mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)(4 * (A_BYTES + C::B_BYTES)));
                        const bool mn = warp == LOAD_A ? a_across(w, high, kb) : b_across(w, high, kb);
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t dst = warp == LOAD_A ? to + k * A_BYTES : to + 2 * A_BYTES + k * C::B_BYTES;
                            const int at = warp == LOAD_A ? m : n;
                            if (!mn) {
                                tma_load_3d_pair(dst, along + k, bar, kb * 64, at, w.e);
                            } else {
                                tma_load_3d_pair(dst, cross + k, bar, at, kb * 64, w.e);
                                if (warp == LOAD_A || W == 256) tma_load_3d_pair(dst + 8192, cross + k, bar, at + 64, kb * 64, w.e);
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
        } else if (warp == MMA && leader) {
            // ------------------------------------------------------------ MMA
            const uint32_t a_at = (smem_u32(smem) >> 4) & 0x3FFFu, b_at = ((smem_u32(smem) + 2 * A_BYTES) >> 4) & 0x3FFFu;
            const uint32_t desc_hi = (uint32_t)(smem_desc_sw128(0, 0, 1024) >> 32);
            uint32_t s = 0, ph = 0, use = 0;
            int phase = 0;
            bool ok = true, issued = false;
            for (int i = pair; i < total && ok; i += npairs) {
                const Work w = work_at<W>(p, i, phase);
                for (int left = w.kb1 - w.kb0; left > 0 && ok;) {
                    const uint32_t b = use & 1, bph = (use >> 1) & 1, d = tmem_base + b * 256;
                    ++use;
                    ok = __all_sync(0xffffffffu, wait_cluster(tempty0 + 8 * b, bph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t acc = 0;
                    const int end = left > p.segment ? left - p.segment : 0;
                    for (; left > end; --left) {
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                        if (!ok) break;
                        const bool a_mn = a_across(w, high, w.kb1 - left), b_mn = b_across(w, high, w.kb1 - left);
                        // fp16 operands, fp32 sums; a 16-deep step in 16 bytes; the leading offset of the descriptors
                        const uint32_t id = (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(w.n >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
                        const uint32_t a_step = a_mn ? 128 : 2, b_step = b_mn ? 128 : 2, a_lead = (a_mn ? 8192u >> 4 : 1u) << 16, b_lead = (b_mn ? 8192u >> 4 : 1u) << 16;
                        const uint32_t ad = (a_at + s * (C::STAGE >> 4)) | a_lead, bd = (b_at + s * (C::STAGE >> 4)) | b_lead;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_pair_elect(d, ad + a_step * kk, desc_hi, bd + (C::B_BYTES >> 4) + b_step * kk, desc_hi, id, acc);
                            acc = 1;
                            mma_pair_elect(d, ad + (A_BYTES >> 4) + a_step * kk, desc_hi, bd + b_step * kk, desc_hi, id, acc);
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) mma_pair_elect(d, ad + a_step * kk, desc_hi, bd + b_step * kk, desc_hi, id, acc);
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
            __syncwarp();
        }
    }

    // no remote arrive or MMA may target a CTA that has left
    cluster_sync_all();
    if (warp == MMA) {
        tc_fence_after();
        tmem_dealloc2(tmem_base, 512);
    }
}

template <int W>
cudaError_t prepare_kernel() {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && attr_set[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(orth_kernel<W>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<W>());
    if (e == cudaSuccess && dev >= 0 && dev < 64) attr_set[dev] = true;
    return e;
}
template <int W>
cudaError_t launch_steps(const OrthParams &p, int pairs, cudaStream_t s) {
    const cudaError_t e = prepare_kernel<W>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<W>();
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeCooperative;  // the pairs wait for one another: all of them are resident
    attr.val.cooperative = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, orth_kernel<W>, p);
}

// ---- what comes before the products --------------------------------------------
constexpr int NT = 256;

// A thread's places in a matrix, V elements each: every (blocks x NT)-th.  (With a 64-bit division for each place the norm of 4 of
// 2048 x 1024 took 17 us instead of 14.)
struct Places {
    int r, c, per_row, rows_on, on;
    __device__ __forceinline__ Places(const OrthPrepParams &p, int v) {
        per_row = (p.cols + v - 1) / v;  // (v divides cols where v > 1)
        const uint32_t first = blockIdx.x * NT + threadIdx.x, step = gridDim.x * NT;
        r = (int)(first / (uint32_t)per_row);
        c = (int)(first - (uint32_t)r * (uint32_t)per_row);
        rows_on = (int)(step / (uint32_t)per_row);
        on = (int)(step - (uint32_t)rows_on * (uint32_t)per_row);
    }
    __device__ __forceinline__ void next() {
        r += rows_on;
        c += on;
        if (c >= per_row) {
            c -= per_row;
            ++r;
        }
    }
};

// Squares of u, summed by block; the momentum is updated on the way.  u = g without momentum, else m' = beta m + g and u =
// g + beta m' (nesterov) or m'.
template <int V, bool LINES, bool BF16>
__global__ void __launch_bounds__(NT) orth_norm_kernel(const OrthPrepParams p) {
    __shared__ double part[NT / 32][2];
    pdl_next();
    pdl_wait();
    const int e = blockIdx.y;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.done[e] = 0;
    SquareSum sum = {0.f, 0.f, 0.0};
    for (Places places(p, V); places.r < p.rows; places.next()) {
        const int r = places.r, c = places.c * V;
        const int64_t at = (int64_t)e * p.ls + (int64_t)r * p.ld + c;
        float g[V], m[V];
        load_v<V, LINES, BF16>(p.grad, at, g);
        if (p.momentum) {
            const int64_t to = ((int64_t)e * p.rows + r) * p.cols + c;
            load_v<V, LINES, false>(p.momentum, to, m);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                m[k] = fmaf(p.beta, m[k], g[k]);
                g[k] = p.nesterov ? fmaf(p.beta, m[k], g[k]) : m[k];
            }
            store_v<V, LINES, false>(p.momentum, to, m);
        }
        sum.add(g);
    }
    sum.join();
    if (threadIdx.x % 32 == 0) {
        part[threadIdx.x / 32][0] = (double)sum.safe;
        part[threadIdx.x / 32][1] = sum.rest;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        double s = 0.0;
        for (int i = 0; i < NT / 32; ++i) s += part[i][threadIdx.x];
        p.partial[((int64_t)e * gridDim.x + blockIdx.x) * 2 + threadIdx.x] = s;
    }
}

// X = u 2^10 / |u| as hi + lo.  A matrix of zeros stays one; one whose norm is not finite becomes NaN throughout.
template <int V, bool LINES, bool BF16>
__global__ void __launch_bounds__(NT) orth_split_kernel(const OrthPrepParams p) {
    __shared__ float factor[3];
    pdl_next();
    pdl_wait();
    const int e = blockIdx.y;
    if (threadIdx.x < 32) {
        double s = 0.0, rest = 0.0;
        for (int i = threadIdx.x; i < p.parts; i += 32) {
            s += p.partial[((int64_t)e * p.parts + i) * 2];
            rest += p.partial[((int64_t)e * p.parts + i) * 2 + 1];
        }
        SquareSum sum = {0.f, 0.f, s + rest};
        sum.join();
        if (threadIdx.x == 0) orth_factors(sum, factor[0], factor[1], factor[2]);
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1], f2 = factor[2];
    for (Places places(p, V); places.r < p.rows; places.next()) {
        const int r = places.r, c = places.c * V;
        const int64_t at = (int64_t)e * p.ls + (int64_t)r * p.ld + c;
        float g[V], m[V];
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = 0.f;
        if (!p.momentum || p.nesterov) load_v<V, LINES, BF16>(p.grad, at, g);
        if (p.momentum) {
            load_v<V, LINES, false>(p.momentum, ((int64_t)e * p.rows + r) * p.cols + c, m);
#pragma unroll
            for (int k = 0; k < V; ++k) g[k] = p.nesterov ? fmaf(p.beta, m[k], g[k]) : m[k];
        }
#pragma unroll
        for (int k = 0; k < V; ++k) g[k] = g[k] * f0 * f1 * f2;
        const int64_t to = ((int64_t)e * p.rows + r) * p.pitch + c;
        if constexpr (V == 4) {
            *reinterpret_cast<uint2 *>(p.hi + to) = make_uint2(pack_hi(g[0], g[1]), pack_hi(g[2], g[3]));
            *reinterpret_cast<uint2 *>(p.lo + to) = make_uint2(pack_lo(g[0], g[1]), pack_lo(g[2], g[3]));
        } else {
            const __half h = __float2half_rn(g[0]);
            p.hi[to] = h;
            p.lo[to] = __float2half_rn(g[0] - __half2float(h));
        }
    }
}

template <int V, bool LINES, bool BF16>
cudaError_t launch_prep(const OrthPrepParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.parts, (unsigned)p.batch);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, orth_norm_kernel<V, LINES, BF16>, p);
    return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, orth_split_kernel<V, LINES, BF16>, p);
}

}  // namespace

cudaError_t launch_orth_prep(const OrthPrepParams &p, cudaStream_t s) {
    const bool lines = rows_on_lines(p.bf16, {p.grad}, {p.momentum}, nullptr, p.ld | p.ls);
    if (p.cols % 4) return p.bf16 ? launch_prep<1, false, true>(p, s) : launch_prep<1, false, false>(p, s);
    if (lines) return p.bf16 ? launch_prep<4, true, true>(p, s) : launch_prep<4, true, false>(p, s);
    return p.bf16 ? launch_prep<4, false, true>(p, s) : launch_prep<4, false, false>(p, s);
}

// Pairs of SMs that can be resident at once.
int orth_pairs(int num_sms) {
    if (prepare_kernel<256>() != cudaSuccess || prepare_kernel<128>() != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(num_sms & ~1));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem_bytes<256>() > smem_bytes<128>() ? smem_bytes<256>() : smem_bytes<128>();
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (prepare_kernel<256>() != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, orth_kernel<256>, &cfg) != cudaSuccess) return 0;
    return n < num_sms / 2 ? n : num_sms / 2;
}

cudaError_t launch_orth_steps(const OrthParams &p, bool wide, int pairs, cudaStream_t s) {
    return wide ? launch_steps<256>(p, pairs, s) : launch_steps<128>(p, pairs, s);
}

}  // namespace cbd
