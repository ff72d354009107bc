// orth_sm103.cu -- Newton-Schulz orthogonalisation of matrices: X <- a X + b (X X^T) X + c (X X^T)^2 X, `steps` times, from
// X = u / |u|_F.
//
// With the smaller side as the Gram side (X^T X for high matrices, from the right):
//   gram     A = X X^T                  or X^T X
//   square   B = c A A + b A + a I
//   product  X' = B X                   or X B
// three products a step, each a launch; the first two are symmetric: tiles below the diagonal blocks are not
// computed but written transposed from those above.
//
// Precision.  A small singular value grows by a = 3.44 a step, and with it what a rounding has put beside it: one fp16
// or bf16 product each leaves 0.4 to 4 % (simulated on matrices of falling spectrum), above what a bf16 result holds.
// So the matrices between the products are pairs of fp16, hi + lo (22 bits), times 2^10 (the polynomial B 2^8) so that lo
// stays a normal number; a product is hi hi + hi lo + lo hi, on the tensor cores in fp32.  (fp16 rather than bf16: 22 bits
// instead of 16 at the same rate.  Singular values stay below 1.3 with the usual coefficients; B may reach 255, which the
// host's bound of 32 on each coefficient keeps below singular values of 1.5.)  The accumulator truncates, about 2^-26 of the sum with each instruction; a new one is begun every SEGMENT k-blocks and
// added in fp32 registers, under the other accumulator's MMAs.
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
#include "tc_common.cuh"
#include "tc_pair.cuh"
#include "train.h"

namespace cbd {

namespace {

constexpr int EPI = 8, LOAD_A = 8, LOAD_B = 9, MMA = 10, THREADS = 512;
constexpr int A_BYTES = 128 * 64 * 2;  // of one plane of a stage
constexpr int OUT_BYTES = EPI * 4096;
constexpr int SEGMENT = 2;  // k-blocks (of 64) of one accumulator

template <int W>
struct Cfg {
    static constexpr int B_BYTES = W / 2 * 64 * 2;  // one CTA's half of the tile's columns
    static constexpr int STAGE = 2 * (A_BYTES + B_BYTES);
    static constexpr int S = W == 256 ? 3 : 4;
};
struct Bars {
    uint64_t full[4], empty[4], tfull[2], tempty[2];
    uint32_t tmem;
    int32_t abort;
};
template <int W>
constexpr int smem_bytes() {
    return 1024 + Cfg<W>::S * Cfg<W>::STAGE + OUT_BYTES + (int)sizeof(Bars);
}
static_assert(smem_bytes<256>() <= 232448 && smem_bytes<128>() <= 232448, "shared memory of one CTA");

struct Tile {
    int e, m0, n0, n;  // matrix, first row and column, columns (a multiple of 32)
};
template <int W>
__device__ __forceinline__ Tile tile_at(const OrthGemmParams &p, int t) {
    Tile r;
    const int nt = (p.N + W - 1) / W;
    r.e = t / p.tiles;
    int l = t - r.e * p.tiles, tm, tn;
    if (p.symmetric) {  // from the diagonal block on
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
    r.m0 = tm * 256;
    r.n0 = tn * W;
    r.n = min(W, (p.N - r.n0 + 31) & ~31);
    return r;
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

// One warp's 32 rows x COLS columns of a tile, in registers, to the planes hi and lo (and transposed).
template <int COLS>
__device__ __forceinline__ void store_planes(const OrthGemmParams &p, const float (&v)[COLS], uint8_t *slab, int e, int row, int col, bool mirror, int lane) {
    const uint32_t sb = smem_u32(slab);
#pragma unroll
    for (int g = 0; g < COLS / 64; ++g)
#pragma unroll
        for (int plane = 0; plane < 2; ++plane) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = v[g * 64 + q * 8 + 2 * i], y = v[g * 64 + q * 8 + 2 * i + 1];
                    w[i] = plane ? pack_lo(x, y) : pack_hi(x, y);
                }
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (uint32_t)lane * 128u + (((uint32_t)q ^ (lane & 7)) << 4)), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row < p.M && col + g * 64 < p.N) store_box(&p.out[plane], sb, col + g * 64, row, e);
            if (!mirror) continue;
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                const float x = v[g * 64 + 2 * q], y = v[g * 64 + 2 * q + 1];
                const uint32_t w = plane ? pack_lo(x, y) : pack_hi(x, y);
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(sb + (uint32_t)(2 * q) * 64u + (uint32_t)lane * 2u), "h"((uint16_t)w) : "memory");
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(sb + (uint32_t)(2 * q + 1) * 64u + (uint32_t)lane * 2u), "h"((uint16_t)(w >> 16)) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && row < p.M && col + g * 64 < p.N) store_box(&p.out_t[plane], sb, row, col + g * 64, e);
        }
}

// The same to the caller's tensors: the result itself, or the step on the weights.
template <int COLS>
__device__ __forceinline__ void store_result(const OrthGemmParams &p, const float (&v)[COLS], uint8_t *slab, int e, int row, int col, int lane) {
    const uint32_t sb = smem_u32(slab);
#pragma unroll
    for (int g = 0; g < COLS / 32; ++g) {
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sb + (uint32_t)lane * 128u + (((uint32_t)q ^ (lane & 7)) << 4)),
                         "f"(v[g * 32 + 4 * q]), "f"(v[g * 32 + 4 * q + 1]), "f"(v[g * 32 + 4 * q + 2]), "f"(v[g * 32 + 4 * q + 3])
                         : "memory");
        __syncwarp();
        const int c = col + g * 32 + lane;
        if (c >= p.N) continue;
        for (int r0 = 0; r0 < 32 && row + r0 < p.M; r0 += 8) {
            float x[8], w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = r0 + i;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[i]) : "r"(sb + (uint32_t)r * 128u + (((uint32_t)(lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4u) : "memory");
            }
            if (p.weight) {
                const int64_t at = (int64_t)e * p.lse + (int64_t)(row + r0) * p.ldo + c;
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = row + r0 + i < p.M ? p.weight[at + i * p.ldo] : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (row + r0 + i >= p.M) break;
                    const float n = fmaf(-p.rate, x[i], w[i] * p.keep);
                    p.weight[at + i * p.ldo] = n;
                    if (p.copy) p.copy[at + i * p.ldo] = __float2bfloat16_rn(n);
                }
            } else {
                const int64_t at = (int64_t)e * p.lse + (int64_t)(row + r0) * p.ldo + c;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (row + r0 + i >= p.M) break;
                    if (p.bf16)
                        static_cast<__nv_bfloat16 *>(p.result)[at + i * p.ldo] = __float2bfloat16_rn(x[i]);
                    else
                        static_cast<float *>(p.result)[at + i * p.ldo] = x[i];
                }
            }
        }
    }
}

template <int W, bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) orth_gemm_kernel(const __grid_constant__ OrthGemmParams p) {
    using C = Cfg<W>;
    constexpr int S = C::S, COLS = W / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *stage = smem + S * C::STAGE;
    Bars &bars = *reinterpret_cast<Bars *>(stage + OUT_BYTES);
    volatile int32_t *abort_flag = &bars.abort;

    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const uint32_t full0 = smem_u32(bars.full), empty0 = smem_u32(bars.empty), tfull0 = smem_u32(bars.tfull), tempty0 = smem_u32(bars.tempty);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;
    const int kblocks = (p.K + 63) / 64, total = p.batch * p.tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull0 + 8 * b, 1);
            mbar_init(tempty0 + 8 * b, 2 * EPI);  // epilogue warps of both CTAs
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == MMA) {
        tmem_alloc2(smem_u32(&bars.tmem), 512);
        tc_fence_before();
    }
    if ((warp == LOAD_A || warp == LOAD_B) && lane == 0)
        for (int i = 0; i < 2; ++i) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(warp == LOAD_A ? &p.a[i] : &p.b[i])) : "memory");
    cluster_sync_all();
    tc_fence_after();
    pdl_next();
    pdl_wait();
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
        uint32_t use = 0;
        bool ok = true;
        for (int t = pair; t < total; t += npairs) {
            const Tile w = tile_at<W>(p, t);
            const int row = w.m0 + (int)rank * 128 + (warp % 4) * 32, col0 = (warp / 4) * COLS, col = w.n0 + col0;
            float sum[COLS];
#pragma unroll
            for (int q = 0; q < COLS; ++q) sum[q] = 0.f;
            for (int left = kblocks; left > 0; left -= SEGMENT, ++use) {
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
            if (!ok) continue;
            if (p.old[0]) {
                // square: c sum + b A + a on the diagonal
                const int r = row + lane;
                const int64_t at = ((int64_t)w.e * p.M + r) * p.ld_old;
#pragma unroll
                for (int q = 0; q < COLS / 8; ++q) {
                    const int c = col + q * 8;
                    uint4 h = make_uint4(0u, 0u, 0u, 0u), l = h;
                    if (r < p.M && c < p.ld_old) {
                        h = *reinterpret_cast<const uint4 *>(p.old[0] + at + c);
                        l = *reinterpret_cast<const uint4 *>(p.old[1] + at + c);
                    }
                    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&hw[i])), y = __half22float2(*reinterpret_cast<const __half2 *>(&lw[i]));
                        float &s0 = sum[q * 8 + 2 * i], &s1 = sum[q * 8 + 2 * i + 1];
                        s0 = fmaf(p.mul, s0, p.mul_old * (x.x + y.x)) + (r == c + 2 * i ? p.diagonal : 0.f);
                        s1 = fmaf(p.mul, s1, p.mul_old * (x.y + y.y)) + (r == c + 2 * i + 1 ? p.diagonal : 0.f);
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < COLS; ++q) sum[q] *= p.mul;
            }
            if (p.final)
                store_result<COLS>(p, sum, slab, w.e, row, col, lane);
            else
                store_planes<COLS>(p, sum, slab, w.e, row, col, p.symmetric && w.n0 >= w.m0 + 256, lane);
        }
        if (lane == 0) bulk_wait_all();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == LOAD_A || warp == LOAD_B) {
            // ------------------------------------------------------------ loads
            if (lane == 0) {
                const uint32_t full_leader0 = mapa_shared(full0, 0);
                const int planes = p.terms == 1 ? 1 : 2;
                uint32_t it = 0;
                bool ok = true, issued = false;
                for (int t = pair; t < total && ok; t += npairs) {
                    const Tile w = tile_at<W>(p, t);
                    const int m = w.m0 + (int)rank * 128, n = w.n0 + (int)rank * (w.n / 2);
                    for (int kb = 0; kb < kblocks; ++kb, ++it) {
                        const uint32_t s = it % S, ph = (it / S) & 1;
                        if (!mbar_wait_bounded(empty0 + 8 * s, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer)) {
                            ok = false;
                            break;
                        }
                        const uint32_t bar = full_leader0 + 8 * s, to = smem_u32(smem + s * C::STAGE);
                        if (warp == LOAD_A) {
                            if (leader) mbar_arrive_expect_tx(full0 + 8 * s, (uint32_t)(2 * planes * (A_BYTES + C::B_BYTES)));
                            for (int i = 0; i < planes; ++i) {
                                const uint32_t dst = to + i * A_BYTES;
                                if constexpr (A_MN) {
                                    tma_load_3d_pair(dst, &p.a[i], bar, m, kb * 64, w.e);
                                    tma_load_3d_pair(dst + 8192, &p.a[i], bar, m + 64, kb * 64, w.e);
                                } else {
                                    tma_load_3d_pair(dst, &p.a[i], bar, kb * 64, m, w.e);
                                }
                            }
                        } else {
                            for (int i = 0; i < planes; ++i) {
                                const uint32_t dst = to + 2 * A_BYTES + i * C::B_BYTES;
                                if constexpr (B_MN) {
                                    for (int h = 0; h < W / 128; ++h) tma_load_3d_pair(dst + 8192 * h, &p.b[i], bar, n + 64 * h, kb * 64, w.e);
                                } else {
                                    tma_load_3d_pair(dst, &p.b[i], bar, kb * 64, n, w.e);
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
        } else if (warp == MMA && leader) {
            // ------------------------------------------------------------ MMA
            constexpr uint32_t A_STEP = A_MN ? 128 : 2, B_STEP = B_MN ? 128 : 2;  // a 16-deep step, in 16 bytes
            const uint32_t idesc0 = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(256 >> 4) << 24);  // fp16 operands, fp32 sums
            const uint64_t a_desc0 = smem_desc_sw128(smem_u32(smem), A_MN ? 8192 : 16, 1024);
            const uint64_t b_desc0 = smem_desc_sw128(smem_u32(smem) + 2 * A_BYTES, B_MN ? 8192 : 16, 1024);
            const uint32_t a_lo = (uint32_t)a_desc0, a_hi = (uint32_t)(a_desc0 >> 32), b_lo = (uint32_t)b_desc0, b_hi = (uint32_t)(b_desc0 >> 32);
            uint32_t s = 0, ph = 0, use = 0;
            bool ok = true, issued = false;
            for (int t = pair; t < total && ok; t += npairs) {
                const uint32_t id = idesc0 | ((uint32_t)(tile_at<W>(p, t).n >> 3) << 17);
                for (int left = kblocks; left > 0 && ok;) {
                    const uint32_t b = use & 1, bph = (use >> 1) & 1, d = tmem_base + b * 256;
                    ++use;
                    ok = __all_sync(0xffffffffu, wait_cluster(tempty0 + 8 * b, bph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t acc = 0;
                    const int end = left > SEGMENT ? left - SEGMENT : 0;
                    for (; left > end; --left) {
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(full0 + 8 * s, ph, p.wait_budget, abort_flag, p.status, kDevTimeoutMma));
                        if (!ok) break;
                        const uint32_t ad = a_lo + s * (C::STAGE >> 4), bd = b_lo + s * (C::STAGE >> 4);
                        if (p.terms > 1) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                mma_pair_elect(d, ad + A_STEP * kk, a_hi, bd + (C::B_BYTES >> 4) + B_STEP * kk, b_hi, id, acc);
                                acc = 1;
                                mma_pair_elect(d, ad + (A_BYTES >> 4) + A_STEP * kk, a_hi, bd + B_STEP * kk, b_hi, id, acc);
                            }
                        }
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            mma_pair_elect(d, ad + A_STEP * kk, a_hi, bd + B_STEP * kk, b_hi, id, acc);
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

template <int W, bool A_MN, bool B_MN>
cudaError_t launch_gemm(const OrthGemmParams &p, int num_sms, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(orth_gemm_kernel<W, A_MN, B_MN>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<W>());
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int64_t tiles = (int64_t)p.batch * p.tiles;
    const int pairs = num_sms / 2 > 1 ? num_sms / 2 : 1;
    return launch_early(orth_gemm_kernel<W, A_MN, B_MN>, 2 * (int)(tiles < pairs ? tiles : pairs), THREADS, smem_bytes<W>(), s, p);
}

// ---- what comes before the products --------------------------------------------
// Elements four at a time where every row starts on four elements' bytes, else one at a time.
__device__ __forceinline__ float load1(const void *x, int64_t i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]) : static_cast<const float *>(x)[i];
}
__device__ __forceinline__ float4 load4(const void *x, int64_t i, bool bf16) {
    if (!bf16) return *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(x) + i);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

constexpr int NT = 256;

// Squares of u, summed by block; the momentum is updated on the way.  u = g without momentum, else m' = beta m + g and u =
// g + beta m' (nesterov) or m'.  (Summed in fp64, four squares at a time in fp32 where they are far from its ends: a
// conversion and an addition of fp64 for each element would take longer than the memory.)
template <int V>
__global__ void __launch_bounds__(NT) orth_norm_kernel(const OrthPrepParams p) {
    __shared__ double part[NT / 32];
    pdl_next();
    pdl_wait();
    const int e = blockIdx.y;
    const int per_row = (p.cols + V - 1) / V;  // (V divides cols where V > 1)
    const int64_t items = (int64_t)p.rows * per_row;
    double sum = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < items; i += (int64_t)gridDim.x * NT) {
        const int r = (int)(i / per_row), c = (int)(i - (int64_t)r * per_row) * V;
        const int64_t at = (int64_t)e * p.ls + (int64_t)r * p.ld + c;
        float g[V], m[V];
        if constexpr (V == 4) {
            const float4 x = load4(p.grad, at, p.bf16);
            g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w;
        } else {
            g[0] = load1(p.grad, at, p.bf16);
        }
        if (p.momentum) {
            float *to = p.momentum + ((int64_t)e * p.rows + r) * p.cols + c;
            if constexpr (V == 4)
                *reinterpret_cast<float4 *>(m) = *reinterpret_cast<const float4 *>(to);
            else
                m[0] = *to;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                m[k] = fmaf(p.beta, m[k], g[k]);
                g[k] = p.nesterov ? fmaf(p.beta, m[k], g[k]) : m[k];
            }
            if constexpr (V == 4)
                *reinterpret_cast<float4 *>(to) = *reinterpret_cast<const float4 *>(m);
            else
                *to = m[0];
        }
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) q = fmaf(g[k], g[k], q);
        if (q > 0x1p-60f && q < 0x1p120f) {  // far from both ends of fp32, each square above 2^-24 of q among them
            sum += (double)q;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) sum += (double)g[k] * (double)g[k];
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < NT / 32; ++i) s += part[i];
        p.partial[(int64_t)e * gridDim.x + blockIdx.x] = s;
    }
}

// X = u 2^10 / |u| as hi + lo.  A matrix of zeros stays one; one whose norm is not finite becomes NaN throughout.
template <int V>
__global__ void __launch_bounds__(NT) orth_split_kernel(const OrthPrepParams p) {
    __shared__ float factor[3];
    pdl_next();
    pdl_wait();
    const int e = blockIdx.y;
    if (threadIdx.x < 32) {
        double s = 0.0;
        for (int i = threadIdx.x; i < p.parts; i += 32) s += p.partial[(int64_t)e * p.parts + i];
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (threadIdx.x == 0) {
            const double n = sqrt(s);
            if (!isfinite(n)) {
                factor[0] = factor[1] = factor[2] = __uint_as_float(0x7fffffffu);
            } else if (n == 0.0) {
                factor[0] = factor[1] = factor[2] = 0.f;
            } else {
                // 2^10 / n in three factors that neither overflow nor underflow: n is anywhere from 2^-149 on
                int x;
                const double f = frexp(n, &x);
                const int k = 10 - x;
                factor[0] = ldexpf(1.f, k / 2);
                factor[1] = ldexpf(1.f, k - k / 2);
                factor[2] = (float)(1.0 / f);
            }
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1], f2 = factor[2];
    const int per_row = (p.cols + V - 1) / V;
    const int64_t items = (int64_t)p.rows * per_row;
    for (int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x; i < items; i += (int64_t)gridDim.x * NT) {
        const int r = (int)(i / per_row), c = (int)(i - (int64_t)r * per_row) * V;
        const int64_t at = (int64_t)e * p.ls + (int64_t)r * p.ld + c;
        float g[V];
        const float *from = p.momentum ? p.momentum + ((int64_t)e * p.rows + r) * p.cols + c : nullptr;
        const bool grad = !from || p.nesterov;
        if constexpr (V == 4) {
            const float4 x = grad ? load4(p.grad, at, p.bf16) : make_float4(0.f, 0.f, 0.f, 0.f);
            g[0] = x.x, g[1] = x.y, g[2] = x.z, g[3] = x.w;
        } else {
            g[0] = grad ? load1(p.grad, at, p.bf16) : 0.f;
        }
        if (from) {
            float m[V];
            if constexpr (V == 4)
                *reinterpret_cast<float4 *>(m) = *reinterpret_cast<const float4 *>(from);
            else
                m[0] = *from;
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

}  // namespace

cudaError_t launch_orth_prep(const OrthPrepParams &p, bool by_four, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.parts, (unsigned)p.batch);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = by_four ? cudaLaunchKernelEx(&cfg, orth_norm_kernel<4>, p) : cudaLaunchKernelEx(&cfg, orth_norm_kernel<1>, p);
    if (e != cudaSuccess) return e;
    return by_four ? cudaLaunchKernelEx(&cfg, orth_split_kernel<4>, p) : cudaLaunchKernelEx(&cfg, orth_split_kernel<1>, p);
}

cudaError_t launch_orth_gemm(const OrthGemmParams &p, bool a_mn, bool b_mn, bool wide, int num_sms, cudaStream_t s) {
    if (wide) return a_mn ? launch_gemm<256, true, true>(p, num_sms, s) : b_mn ? launch_gemm<256, false, true>(p, num_sms, s) : launch_gemm<256, false, false>(p, num_sms, s);
    return a_mn ? launch_gemm<128, true, true>(p, num_sms, s) : b_mn ? launch_gemm<128, false, true>(p, num_sms, s) : launch_gemm<128, false, false>(p, num_sms, s);
}

}  // namespace cbd
