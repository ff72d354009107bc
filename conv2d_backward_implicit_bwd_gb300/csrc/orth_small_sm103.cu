// orth_small_sm103.cu -- Newton-Schulz orthogonalisation of matrices whose smaller side is at most 128, in one launch:
// the iteration of orth_sm103.cu with everything between the first read and the last write in shared memory.
//
// A matrix is held with its smaller side as rows, [128][n], cut into slices of at most 256 columns over the CTAs of a
// cluster (one CTA where n <= 256).  Per step, on a CTA's tensor core (tcgen05, 128 x 128 and 128 x slice):
//   A = X X^T     both operands the slice, contraction along it; the cluster's CTAs add their parts in order through
//                 distributed shared memory
//   B = c A A + b A + a I   each CTA for itself
//   X = B X       in place: the product is in tensor memory before the slice is written again
// The planes hi and lo of a slice, [128 rows][64 columns] blocks of 128-byte swizzled lines, are the K-major operand of
// the first product and the MN-major operand of the last.  Rows and columns beyond the matrix are zeros and stay so
// (B's last rows hold a on the diagonal, which multiplies rows of zeros).
//
// What bounds it is the chain of fifteen products: at these sizes each is a fraction of a microsecond of work, and a tile
// through global memory and a flag costs 7.7 us (100 x 131, 15 products: 117 us in the kernel for large matrices).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "device_util.cuh"
#include "internal.h"
#include "tc_common.cuh"
#include "train.h"

namespace cbd {

namespace {

constexpr int NT = 512, WARPS = NT / 32;
constexpr int BLOCK = 128 * 128;            // bytes of 128 rows x 64 columns of a plane
constexpr int X_PLANE = 4 * BLOCK, G_PLANE = 2 * BLOCK;
constexpr int SMEM = 1024 + 2 * X_PLANE + 2 * G_PLANE;
static_assert(2 * X_PLANE == 128 * 256 * 4 && 2 * G_PLANE == 128 * 128 * 4, "a slice and a Gram matrix in fp32 fit their planes");

__device__ __forceinline__ uint32_t half_bits(float x) {
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_hi(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack_lo(float x, float y) {
    const float2 h = __half22float2(__floats2half2_rn(x, y));
    return pack_hi(x - h.x, y - h.y);
}
__device__ __forceinline__ float2 unpack(uint32_t h, uint32_t l) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h)), y = __half22float2(*reinterpret_cast<const __half2 *>(&l));
    return make_float2(x.x + y.x, x.y + y.y);
}
// byte of the 16 bytes that hold columns [c, c + 8) of row r, c a multiple of 8, within a plane
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return (uint32_t)(c >> 6) * BLOCK + (uint32_t)r * 128u + (((uint32_t)(c >> 3) ^ (uint32_t)r) & 7u) * 16u; }
// float of row r, column c in an area of `width` floats a row, 16-byte chunks swapped so that a column's reads spread
__device__ __forceinline__ uint32_t float_at(int r, int c, int width) { return (uint32_t)r * (uint32_t)width + ((((uint32_t)c >> 2) ^ ((uint32_t)r & 7u)) << 2) + ((uint32_t)c & 3u); }
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t a_lead, uint32_t b, uint32_t b_lead, uint32_t hi, uint32_t idesc, uint32_t acc) {
    tc_mma(d, (uint64_t)hi << 32 | (((a >> 4) & 0x3FFFu) | a_lead << 16), (uint64_t)hi << 32 | (((b >> 4) & 0x3FFFu) | b_lead << 16), idesc, acc);
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ float load1(const void *x, int64_t i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]) : static_cast<const float *>(x)[i];
}

__global__ void __launch_bounds__(NT, 1) orth_small_kernel(const OrthSmallParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sx = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)), *sg = sx + 2 * X_PLANE;
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_;
    __shared__ double partial[WARPS], mine_sum;
    __shared__ float factor[3];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, c = p.cluster;
    const int rank = c > 1 ? (int)cluster_ctarank() : 0, e = blockIdx.x / c;
    const bool high = p.rows > p.cols;
    const int g = min(p.rows, p.cols), n = max(p.rows, p.cols), width = p.slice;
    const int col0 = rank * width, valid = max(0, min(width, n - col0));  // the slice's columns
    const uint32_t bar_at = smem_u32(&bar), x_at = smem_u32(sx), g_at = smem_u32(sg);
    auto sync_all = [&] {
        if (c > 1)
            cluster_sync_all();
        else
            __syncthreads();
    };
    if (tid == 0) {
        mbar_init(bar_at, 1);
        abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), 256);
    tc_fence_before();
    for (int i = tid; i < 2 * X_PLANE / 16; i += NT) reinterpret_cast<uint4 *>(sx)[i] = make_uint4(0u, 0u, 0u, 0u);
    pdl_next();
    pdl_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // ---- u, its norm, and the planes
    // Element i of the slice: along the caller's rows, so that a warp's loads are neighbours.
    const int inner = high ? g : valid, items = g * valid;
    auto place = [&](int i, int &r, int &cc, int64_t &at, int64_t &at_m) {  // row and column of X; of the caller's tensors
        const int o = i / inner, k = i - o * inner;
        r = high ? k : o;
        cc = high ? o : k;
        const int row = high ? col0 + o : o, col = high ? k : col0 + k;
        at = (int64_t)e * p.ls + (int64_t)row * p.ld + col;
        at_m = ((int64_t)e * p.rows + row) * p.cols + col;
    };
    constexpr int U = 8;
    double sum = 0.0;
    for (int i0 = tid; i0 < items; i0 += U * NT) {
        float x[U], m[U];
        int64_t at_m[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            int r, cc;
            int64_t at;
            place(min(i0 + k * NT, items - 1), r, cc, at, at_m[k]);
            x[k] = load1(p.grad, at, p.in_bf16);
            if (p.momentum) m[k] = p.momentum[at_m[k]];
        }
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * NT >= items) {
                x[k] = 0.f;
                continue;
            }
            if (p.momentum) {
                m[k] = fmaf(p.beta, m[k], x[k]);
                p.momentum[at_m[k]] = m[k];
                x[k] = p.nesterov ? fmaf(p.beta, m[k], x[k]) : m[k];
            }
            q = fmaf(x[k], x[k], q);
        }
        if (q > 0x1p-60f && q < 0x1p120f) {  // far from both ends of fp32
            sum += (double)q;
        } else {
#pragma unroll
            for (int k = 0; k < U; ++k) sum += (double)x[k] * (double)x[k];
        }
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) partial[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.0;
        for (int i = 0; i < WARPS; ++i) sum += partial[i];
        mine_sum = sum;
    }
    sync_all();
    if (tid == 0) {
        sum = 0.0;
        for (int k = 0; k < c; ++k) {
            double x = mine_sum;
            if (c > 1) asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(x) : "r"(mapa_shared(smem_u32(&mine_sum), k)) : "memory");
            sum += x;
        }
        orth_factors(sum, factor);
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1], f2 = factor[2];
    for (int i0 = tid; i0 < items; i0 += U * NT) {
        float x[U];
        uint32_t to[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            int r, cc;
            int64_t at, at_m;
            place(min(i0 + k * NT, items - 1), r, cc, at, at_m);
            to[k] = chunk_at(r, cc & ~7) + (uint32_t)(cc & 7) * 2u;
            x[k] = p.momentum && !p.nesterov ? 0.f : load1(p.grad, at, p.in_bf16);
            if (p.momentum) {
                const float m = p.momentum[at_m];  // (this thread's own)
                x[k] = p.nesterov ? fmaf(p.beta, m, x[k]) : m;
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * NT >= items) break;
            const float v = x[k] * f0 * f1 * f2;
            const uint32_t h = half_bits(v);
            *reinterpret_cast<uint16_t *>(sx + to[k]) = (uint16_t)h;
            const uint16_t hb = (uint16_t)h;
            *reinterpret_cast<uint16_t *>(sx + X_PLANE + to[k]) = (uint16_t)half_bits(v - __half2float(*reinterpret_cast<const __half *>(&hb)));
        }
    }

    // ---- the steps
    // A thread's part of a product: row 32 (warp % 4) + lane, a fourth of the columns.
    const int row = warp % 4 * 32 + lane, part = warp / 4;
    const uint32_t lane_base = tmem + ((uint32_t)(warp % 4 * 32) << 16);
    const uint32_t desc_hi = (uint32_t)(smem_desc_sw128(0, 0, 1024) >> 32);
    uint32_t phase = 0;
    bool ok = true;
    auto product = [&](auto &&issue) {  // by one thread, then waited for by all
        fence_proxy_async();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (tid == 0) {
            issue();
            tc_commit(bar_at);
        }
        if (ok) ok = mbar_wait_bounded(bar_at, phase, p.wait_budget, &abort_, p.status, kDevTimeoutMma);
        phase ^= 1;
        tc_fence_after();
        __syncwarp();
    };
    const int deep = (g + 15) / 16;  // 16-deep steps of a contraction over the smaller side
    for (int step = 0; step < p.steps; ++step) {
        const bool single = step >= p.single_from, final = step + 1 == p.steps;
        const int terms = single ? 1 : 3;
        // gram
        product([&] {
            const uint32_t id = (1u << 4) | (128u >> 3) << 17 | (128u >> 4) << 24;
            uint32_t acc = 0;
            for (int kb = 0; kb < width / 64; ++kb)
                for (int t = terms; t--;)  // the small terms first
                    for (int kk = 0; kk < 4; ++kk, acc = 1)
                        mma(tmem, x_at + (t == 1 ? X_PLANE : 0) + kb * BLOCK + kk * 32, 1, x_at + (t == 2 ? X_PLANE : 0) + kb * BLOCK + kk * 32, 1, desc_hi, id, acc);
        });
        {
            uint32_t v[32];
            tmem_ld32(lane_base + part * 32, v);
            if (c == 1) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = __uint_as_float(v[q * 8 + 2 * i]) * (1.f / kOrthUp), y = __uint_as_float(v[q * 8 + 2 * i + 1]) * (1.f / kOrthUp);
                        h[i] = pack_hi(x, y);
                        l[i] = pack_lo(x, y);
                    }
                    const uint32_t to = chunk_at(row, part * 32 + q * 8);
                    *reinterpret_cast<uint4 *>(sg + to) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(sg + G_PLANE + to) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            } else {
                // this CTA's part, then the sums of 128 / c rows from every CTA, then those to every CTA
                float *f = reinterpret_cast<float *>(sg);
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    *reinterpret_cast<uint4 *>(f + float_at(row, part * 32 + q * 4, 128)) = make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                cluster_sync_all();
                constexpr int MOST = 128 * 32 / 2 / NT;  // chunks of a thread, two CTAs
                const int rows_here = 128 / c;
                float4 s[MOST];
#pragma unroll
                for (int q = 0; q < MOST; ++q) {
                    const int j = q * NT + tid, r = rank * rows_here + j / 32, cc = j % 32 * 4;
                    s[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (j < rows_here * 32) {
                        const uint32_t from = smem_u32(f + float_at(r, cc, 128));
                        for (int k = 0; k < c; ++k) {
                            float4 x;
                            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(mapa_shared(from, k)) : "memory");
                            s[q].x += x.x;
                            s[q].y += x.y;
                            s[q].z += x.z;
                            s[q].w += x.w;
                        }
                    }
                }
                cluster_sync_all();
#pragma unroll
                for (int q = 0; q < MOST; ++q) {
                    const int j = q * NT + tid, r = rank * rows_here + j / 32, cc = j % 32 * 4;
                    if (j < rows_here * 32) {
                        const float m = 1.f / kOrthUp;
                        const uint32_t h0 = pack_hi(s[q].x * m, s[q].y * m), h1 = pack_hi(s[q].z * m, s[q].w * m), l0 = pack_lo(s[q].x * m, s[q].y * m), l1 = pack_lo(s[q].z * m, s[q].w * m);
                        const uint32_t to = g_at + chunk_at(r, cc & ~7) + (uint32_t)(cc & 4) * 2u;
                        for (int k = 0; k < c; ++k) {
                            const uint32_t there = mapa_shared(to, k);
                            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(there), "r"(h0), "r"(h1) : "memory");
                            asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(there + G_PLANE), "r"(l0), "r"(l1) : "memory");
                        }
                    }
                }
                fence_proxy_async();
                cluster_sync_all();
            }
        }
        // square
        product([&] {
            const uint32_t id = (1u << 4) | (128u >> 3) << 17 | (128u >> 4) << 24;
            uint32_t acc = 0;
            for (int t = terms; t--;)
                for (int k = 0; k < deep; ++k, acc = 1) {
                    const uint32_t at = g_at + (k >> 2) * BLOCK + (k & 3) * 32;
                    mma(tmem, at + (t == 1 ? G_PLANE : 0), 1, at + (t == 2 ? G_PLANE : 0), 1, desc_hi, id, acc);
                }
        });
        {
            const float a = p.coef[3 * step] * kOrthUpPoly, b = p.coef[3 * step + 1] * (kOrthUpPoly / kOrthUp), cq = p.coef[3 * step + 2] * (kOrthUpPoly / (kOrthUp * kOrthUp));
            uint32_t v[32];
            tmem_ld32(lane_base + part * 32, v);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int col = part * 32 + q * 8;
                uint4 *at_h = reinterpret_cast<uint4 *>(sg + chunk_at(row, col)), *at_l = reinterpret_cast<uint4 *>(sg + G_PLANE + chunk_at(row, col));
                const uint4 oh = *at_h, ol = *at_l;
                const uint32_t hw[4] = {oh.x, oh.y, oh.z, oh.w}, lw[4] = {ol.x, ol.y, ol.z, ol.w};
                uint32_t h[4], l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 old = unpack(hw[i], lw[i]);
                    const float x = fmaf(cq, __uint_as_float(v[q * 8 + 2 * i]), b * old.x) + (row == col + 2 * i ? a : 0.f);
                    const float y = fmaf(cq, __uint_as_float(v[q * 8 + 2 * i + 1]), b * old.y) + (row == col + 2 * i + 1 ? a : 0.f);
                    h[i] = pack_hi(x, y);
                    l[i] = pack_lo(x, y);
                }
                *at_h = make_uint4(h[0], h[1], h[2], h[3]);
                *at_l = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
        // product
        product([&] {
            const uint32_t id = (1u << 4) | 1u << 16 | (uint32_t)(width >> 3) << 17 | (128u >> 4) << 24;
            uint32_t acc = 0;
            for (int t = terms; t--;)
                for (int k = 0; k < deep; ++k, acc = 1)
                    mma(tmem, g_at + (t == 1 ? G_PLANE : 0) + (k >> 2) * BLOCK + (k & 3) * 32, 1, x_at + (t == 2 ? X_PLANE : 0) + k * 2048, BLOCK >> 4, desc_hi, id, acc);
        });
        const int each = width / 4;  // columns of a thread, a multiple of 16
        const float mul = final ? 1.f / (kOrthUp * kOrthUpPoly) : 1.f / kOrthUpPoly;
        for (int q = 0; q < each; q += 16) {
            uint32_t v[16];
            const int col = part * each + q;
            tmem_ld16(lane_base + col, v);
            if (final) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4 *>(reinterpret_cast<float *>(sx) + float_at(row, col + 4 * i, width)) =
                        make_float4(__uint_as_float(v[4 * i]) * mul, __uint_as_float(v[4 * i + 1]) * mul, __uint_as_float(v[4 * i + 2]) * mul, __uint_as_float(v[4 * i + 3]) * mul);
                continue;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __uint_as_float(v[k * 8 + 2 * i]) * mul, y = __uint_as_float(v[k * 8 + 2 * i + 1]) * mul;
                    h[i] = pack_hi(x, y);
                    l[i] = pack_lo(x, y);
                }
                const uint32_t to = chunk_at(row, col + k * 8);
                *reinterpret_cast<uint4 *>(sx + to) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(sx + X_PLANE + to) = make_uint4(l[0], l[1], l[2], l[3]);
            }
        }
    }

    // ---- the result, along the caller's rows
    tc_fence_before();
    __syncthreads();
    const float *fx = reinterpret_cast<const float *>(sx);
    for (int i0 = tid; ok && i0 < items; i0 += U * NT) {
        float x[U], old[U];
        int64_t at[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            int r, cc;
            int64_t skip;
            const int i = min(i0 + k * NT, items - 1);
            place(i, r, cc, skip, at[k]);
            x[k] = fx[float_at(r, cc, width)];
            if (p.weight)
                old[k] = p.weight[at[k]];
            else
                at[k] = (int64_t)e * p.lse + (int64_t)(high ? col0 + cc : r) * p.ldo + (high ? r : col0 + cc);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k * NT >= items) break;
            if (p.weight) {
                const float w = fmaf(-p.rate, x[k], old[k] * p.keep);
                p.weight[at[k]] = w;
                if (p.copy) p.copy[at[k]] = __float2bfloat16_rn(w);
            } else if (p.out_bf16) {
                static_cast<__nv_bfloat16 *>(p.result)[at[k]] = __float2bfloat16_rn(x[k]);
            } else {
                static_cast<float *>(p.result)[at[k]] = x[k];
            }
        }
    }
    sync_all();  // no CTA of the cluster reads another that has left
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

}  // namespace

cudaError_t launch_orth_small(const OrthSmallParams &p, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(orth_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * p.cluster));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, orth_small_kernel, p);
}

}  // namespace cbd
