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
// through global memory and a flag costs 7.7 us (100 x 131, 15 products: 41 us here, 107 in the kernel for large matrices).  So steps
// are not joined here either: that makes the chain longer.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "device_util.cuh"
#include "internal.h"
#include "rows_io.cuh"
#include "tc_common.cuh"
#include "train.h"

namespace cbd {

namespace {

constexpr int NT = 512, WARPS = NT / 32;
constexpr int BLOCK = 128 * 128;            // bytes of 128 rows x 64 columns of a plane
constexpr int X_PLANE = 4 * BLOCK, G_PLANE = 2 * BLOCK;
constexpr int SMEM = 1024 + 2 * X_PLANE + 2 * G_PLANE;
static_assert(2 * X_PLANE == 128 * 256 * 4 && 2 * G_PLANE == 128 * 128 * 4, "a slice and a Gram matrix in fp32 fit their planes");

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
// One lane of a warp that runs converged issues (a single thread in a branch takes 80 to 100 clocks for each MMA of 64).
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// The low word of a descriptor: 16-byte address and leading offset.
__device__ __forceinline__ uint32_t desc(uint32_t addr, uint32_t lead) { return ((addr >> 4) & 0x3FFFu) | lead << 16; }
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

// V: elements that a thread takes at a time along the caller's rows, by rows_io.cuh.
// (Loads beyond the slice's end take an element inside: with a branch at each the loads waited for one another, 5 thousand
// clocks for 13 thousand elements.)
template <int V, bool LINES, bool BF16>
__global__ void __launch_bounds__(NT, 1) orth_small_kernel(const OrthSmallParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sx = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023)), *sg = sx + 2 * X_PLANE;
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_;
    __shared__ SquareSum partial[WARPS], total;
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
    // (Short code: the start of a launch waits for instructions.)
    const int inner = high ? g : valid, outer = high ? valid : g;  // of the slice: along the caller's rows, across them
    const int row0 = high ? col0 : 0, left = high ? 0 : col0;      // its corner in the caller's matrix
    const int64_t corner = ((int64_t)e * p.rows + row0) * p.cols + left, given = (int64_t)e * p.ls + (int64_t)row0 * p.ld + left;
    if (p.weight)  // needed last, and from memory: on its way to L2 meanwhile
        for (int i = tid; i < outer; i += NT)
            for (int k = 0; k < inner; k += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.weight + corner + (int64_t)i * p.cols + k));
    // The sum of squares, along the caller's rows.
    constexpr int U = 8 / V;  // loads of a thread in flight
    SquareSum sum = {0.f, 0.f, 0.0};
    {
        const int fast = inner / V, items = fast * outer, over = fast ? NT / fast : 0, rest = fast ? NT % fast : 0;
        const int k0 = fast ? tid % fast : 0, o0 = fast ? tid / fast : 0;
        int k = k0, o = o0;
#pragma unroll 1
        for (int i0 = tid; i0 < items; i0 += U * NT) {
            float x[U][V], m[U][V];
            int to[U];  // (a slice of a small matrix)
#pragma unroll
            for (int j = 0; j < U; ++j) {
#pragma unroll
                for (int l = 0; l < V; ++l) x[j][l] = m[j][l] = 0.f;
                const bool there = i0 + j * NT < items;
                to[j] = there ? o * p.cols + k * V : 0;
                load_v<V, LINES, BF16>(p.grad, there ? given + (int64_t)o * p.ld + k * V : given, x[j]);
                if (p.momentum) load_v<V, LINES, false>(p.momentum, corner + to[j], m[j]);
#pragma unroll
                for (int l = 0; l < V; ++l) x[j][l] = there ? x[j][l] : 0.f, m[j][l] = there ? m[j][l] : 0.f;
                o += over;
                k += rest;
                if (k >= fast) {
                    k -= fast;
                    ++o;
                }
            }
            if (p.momentum) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
#pragma unroll
                    for (int l = 0; l < V; ++l) {
                        m[j][l] = fmaf(p.beta, m[j][l], x[j][l]);
                        x[j][l] = p.nesterov ? fmaf(p.beta, m[j][l], x[j][l]) : m[j][l];
                    }
                    if (i0 + j * NT < items) store_v<V, LINES, false>(p.momentum, corner + to[j], m[j]);
                }
            }
            float all[U * V];
#pragma unroll
            for (int j = 0; j < U * V; ++j) all[j] = x[j / V][j % V];
            sum.add(all);
        }
    }
    sum.join();
    if (lane == 0) partial[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = lane < WARPS ? partial[lane] : SquareSum{0.f, 0.f, 0.0};
        sum.join();
        if (lane == 0) total = sum;
    }
    sync_all();
    sum = total;
    if (c > 1) {  // of the whole matrix, in order
        sum = {0.f, 0.f, 0.0};
        for (int k = 0; k < c; ++k) {
            const uint32_t from = mapa_shared(smem_u32(&total), k);
            float x;
            double y;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(from + (uint32_t)offsetof(SquareSum, safe)) : "memory");
            asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(y) : "r"(from + (uint32_t)offsetof(SquareSum, rest)) : "memory");
            sum.safe += x;
            if (y != 0.0) sum.rest += y;
        }
    }
    float f0, f1, f2;
    orth_factors(sum, f0, f1, f2);
    // The planes, eight columns of a row at a time (of V rows where the caller's rows are X's columns), neighbouring threads
    // along the caller's rows.
    {
        const int chunks = (valid + 7) / 8, fast = high ? g / V : chunks, items = high ? fast * chunks : g * chunks;
        auto value = [&](const float x, const float m) { return (p.momentum ? (p.nesterov ? fmaf(p.beta, m, x) : m) : x) * f0 * f1 * f2; };
        auto put = [&](int r, int cc, const float (&x)[8]) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = pack_hi(x[2 * j], x[2 * j + 1]);
                l[j] = pack_lo(x[2 * j], x[2 * j + 1]);
            }
            const uint32_t to = chunk_at(r, cc);
            *reinterpret_cast<uint4 *>(sx + to) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(sx + X_PLANE + to) = make_uint4(l[0], l[1], l[2], l[3]);
        };
        const bool grad = !p.momentum || p.nesterov;
#pragma unroll 1
        for (int i = tid; i < items; i += NT) {
            const int s = i / fast, f = i - s * fast;
            if (high) {
                const int64_t in = given + (int64_t)s * 8 * p.ld + f * V, at = corner + (int64_t)s * 8 * p.cols + f * V;
                float x[8][V], m[8][V];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
#pragma unroll
                    for (int l = 0; l < V; ++l) x[j][l] = m[j][l] = 0.f;
                    const int q = min(j, valid - 1 - s * 8);
                    if (grad) load_v<V, LINES, BF16>(p.grad, in + q * p.ld, x[j]);
                    if (p.momentum) load_fresh<V, LINES>(p.momentum + at + q * p.cols, m[j]);
                }
#pragma unroll
                for (int l = 0; l < V; ++l) {
                    float row[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) row[j] = s * 8 + j < valid ? value(x[j][l], m[j][l]) : 0.f;
                    put(f * V + l, s * 8, row);
                }
            } else {
                const int64_t in = given + (int64_t)s * p.ld + f * 8, at = corner + (int64_t)s * p.cols + f * 8;
                float x[8 / V][V], m[8 / V][V], row[8];
#pragma unroll
                for (int j = 0; j < 8 / V; ++j) {
#pragma unroll
                    for (int l = 0; l < V; ++l) x[j][l] = m[j][l] = 0.f;
                    const int q = min(j * V, valid - V - f * 8);
                    if (grad) load_v<V, LINES, BF16>(p.grad, in + q, x[j]);
                    if (p.momentum) load_fresh<V, LINES>(p.momentum + at + q, m[j]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) row[j] = f * 8 + j < valid ? value(x[j / V][j % V], m[j / V][j % V]) : 0.f;
                put(s, f * 8, row);
            }
        }
    }

    // ---- the steps
    // A thread's part of a product: row 32 (warp % 4) + lane, a fourth of the columns.
    const int row = warp % 4 * 32 + lane, part = warp / 4;
    const uint32_t lane_base = tmem + ((uint32_t)(warp % 4 * 32) << 16);
    const uint32_t desc_hi = (uint32_t)(smem_desc_sw128(0, 0, 1024) >> 32);
    uint32_t phase = 0;
    bool ok = true;
    auto product = [&](auto &&issue) {  // by one warp, then waited for by all
        fence_proxy_async();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 0) {
            __syncwarp();
            issue();
            commit(bar_at);
            __syncwarp();
        }
        if (ok) ok = mbar_wait_bounded(bar_at, phase, p.wait_budget, &abort_, p.status, kDevTimeoutMma);
        phase ^= 1;
        tc_fence_after();
        __syncwarp();
    };
    // What lies beyond the next 16 of the smaller side is zeros in X and never asked for in the Gram matrices.
    const int deep = (g + 15) / 16, gn = deep * 16;  // 16-deep steps of a contraction over the smaller side
    const bool rows_live = warp % 4 * 32 < gn, live = rows_live && part * 32 < gn;
    const int along = max(1, (valid + 15) / 16);  // over the slice
    const uint32_t x_k = desc(x_at, 1), x_mn = desc(x_at, BLOCK >> 4), g_k = desc(g_at, 1);
    // hi hi and, before it, hi lo and lo hi: the small ones first
    auto terms = [&](uint32_t a, uint32_t a_plane, uint32_t b, uint32_t b_plane, int steps, auto &&a_step, auto &&b_step, uint32_t id) {
        uint32_t acc = 0;
#pragma unroll 4
        for (int k = 0; k < steps; ++k, acc = 1) mma(tmem, a + a_step(k), b + b_plane + b_step(k), desc_hi, id, acc);
#pragma unroll 4
        for (int k = 0; k < steps; ++k) mma(tmem, a + a_plane + a_step(k), b + b_step(k), desc_hi, id, 1);
#pragma unroll 4
        for (int k = 0; k < steps; ++k) mma(tmem, a + a_step(k), b + b_step(k), desc_hi, id, 1);
    };
    auto k_step = [](int k) { return (uint32_t)(k >> 2) * (BLOCK >> 4) + (uint32_t)(k & 3) * 2u; };
    auto mn_step = [](int k) { return (uint32_t)k * 128u; };
    constexpr uint32_t XP = X_PLANE >> 4, GP = G_PLANE >> 4;
    auto put_gram = [&](const float (&x)[32]) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t h[4], l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = pack_hi(x[q * 8 + 2 * i], x[q * 8 + 2 * i + 1]);
                l[i] = pack_lo(x[q * 8 + 2 * i], x[q * 8 + 2 * i + 1]);
            }
            const uint32_t to = chunk_at(row, part * 32 + q * 8);
            *reinterpret_cast<uint4 *>(sg + to) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(sg + G_PLANE + to) = make_uint4(l[0], l[1], l[2], l[3]);
        }
    };
    for (int step = 0; step < p.steps; ++step) {
        const bool final = step + 1 == p.steps;
        const uint32_t square_id = (1u << 4) | (uint32_t)(gn >> 3) << 17 | (128u >> 4) << 24;
        // gram
        product([&] { terms(x_k, XP, x_k, XP, along, k_step, k_step, square_id); });
        float old[32];  // this thread's part of A
        if (live) {
            uint32_t v[32];
            tmem_ld32(lane_base + part * 32, v);
#pragma unroll
            for (int q = 0; q < 32; ++q) old[q] = __uint_as_float(v[q]) * (1.f / kOrthUp);
        }
        if (c == 1) {
            if (live) put_gram(old);
        } else {
            // this CTA's part, then the sums of gn / c rows from every CTA, then those to every CTA
            float *f = reinterpret_cast<float *>(sg);
            if (live) {
#pragma unroll
                for (int q = 0; q < 8; ++q) *reinterpret_cast<float4 *>(f + float_at(row, part * 32 + q * 4, 128)) = make_float4(old[4 * q], old[4 * q + 1], old[4 * q + 2], old[4 * q + 3]);
            }
            cluster_sync_all();
            constexpr int MOST = 128 * 32 / 2 / NT;  // chunks of a thread, two CTAs
            const int rows_here = (gn + c - 1) / c, first = rank * rows_here, across = gn / 4, chunks = max(0, min(rows_here, gn - first)) * across;
            float4 s[MOST];
#pragma unroll
            for (int q = 0; q < MOST; ++q) {
                const int j = q * NT + tid, r = first + j / across, cc = j % across * 4;
                s[q] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < chunks) {
                    const uint32_t from = smem_u32(f + float_at(r, cc, 128));
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < c) asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[k].x), "=f"(x[k].y), "=f"(x[k].z), "=f"(x[k].w) : "r"(mapa_shared(from, k)) : "memory");
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (k >= c) break;
                        s[q].x += x[k].x;
                        s[q].y += x[k].y;
                        s[q].z += x[k].z;
                        s[q].w += x[k].w;
                    }
                }
            }
            cluster_sync_all();
#pragma unroll
            for (int q = 0; q < MOST; ++q) {
                const int j = q * NT + tid, r = first + j / across, cc = j % across * 4;
                if (j < chunks) {
                    const uint32_t h0 = pack_hi(s[q].x, s[q].y), h1 = pack_hi(s[q].z, s[q].w), l0 = pack_lo(s[q].x, s[q].y), l1 = pack_lo(s[q].z, s[q].w);
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
            if (live) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 h = *reinterpret_cast<const uint4 *>(sg + chunk_at(row, part * 32 + q * 8)), l = *reinterpret_cast<const uint4 *>(sg + G_PLANE + chunk_at(row, part * 32 + q * 8));
                    const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = unpack(hw[i], lw[i]);
                        old[q * 8 + 2 * i] = x.x;
                        old[q * 8 + 2 * i + 1] = x.y;
                    }
                }
            }
        }
        // square
        product([&] { terms(g_k, GP, g_k, GP, deep, k_step, k_step, square_id); });
        if (live) {
            const float a = p.coef[3 * step] * kOrthUpPoly, b = p.coef[3 * step + 1] * (kOrthUpPoly / kOrthUp), cq = p.coef[3 * step + 2] * (kOrthUpPoly / (kOrthUp * kOrthUp));
            uint32_t v[32];
            tmem_ld32(lane_base + part * 32, v);
#pragma unroll
            for (int q = 0; q < 32; ++q) old[q] = fmaf(cq, __uint_as_float(v[q]), b * old[q]);
            if (warp % 4 == part) {  // the diagonal's warps
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    if (q == lane) old[q] += a;
            }
            put_gram(old);
        }
        // product
        product([&] { terms(g_k, GP, x_mn, XP, deep, k_step, mn_step, (1u << 4) | 1u << 16 | (uint32_t)(width >> 3) << 17 | (128u >> 4) << 24); });
        const int each = width / 4;  // columns of a thread, a multiple of 16
        const float mul = final ? 1.f / (kOrthUp * kOrthUpPoly) : 1.f / kOrthUpPoly;
        for (int q = 0; rows_live && q < each; q += 16) {
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
    {
        const float *fx = reinterpret_cast<const float *>(sx);
        const int64_t ld = p.weight ? p.cols : p.ldo, first = p.weight ? corner : (int64_t)e * p.lse + (int64_t)row0 * p.ldo + left;
        // M vectors of a row or column, `step` apart, those before `many`; every load before the first store
        auto put = [&](auto &x, int64_t at, int64_t step, int many) {
            constexpr int M = sizeof(x) / sizeof(x[0]);
            if (p.weight) {
                float w[M][V];
#pragma unroll
                for (int j = 0; j < M; ++j)
                    load_v<V, LINES, false>(p.weight, at + min(j, many - 1) * step, w[j]);
#pragma unroll
                for (int j = 0; j < M; ++j) {
                    if (j >= many) break;
#pragma unroll
                    for (int l = 0; l < V; ++l) w[j][l] = fmaf(-p.rate, x[j][l], w[j][l] * p.keep);
                    store_v<V, LINES, false>(p.weight, at + j * step, w[j]);
                    if (p.copy) store_v<V, LINES, true>(p.copy, at + j * step, w[j]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < M; ++j)
                    if (j < many) store_v<V, LINES, BF16>(p.result, at + j * step, x[j]);
            }
        };
        // four columns of X at a time, of V rows
        const int chunks = (valid + 3) / 4, fast = high ? g / V : chunks, items = high ? fast * chunks : g * chunks;
#pragma unroll 4
        for (int i = tid; ok && i < items; i += NT) {
            const int s = i / fast, f = i - s * fast;
            if (high) {
                float x[V][4], y[4][V];
#pragma unroll
                for (int l = 0; l < V; ++l) *reinterpret_cast<float4 *>(x[l]) = *reinterpret_cast<const float4 *>(fx + float_at(f * V + l, s * 4, width));
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int l = 0; l < V; ++l) y[j][l] = x[l][j];
                put(y, first + (int64_t)(s * 4) * ld + f * V, ld, valid - s * 4);
            } else {
                float y[4 / V][V];
                *reinterpret_cast<float4 *>(y[0]) = *reinterpret_cast<const float4 *>(fx + float_at(s, f * 4, width));
                put(y, first + (int64_t)s * ld + f * 4, V, (valid - f * 4 + V - 1) / V);
            }
        }
    }
    sync_all();  // no CTA of the cluster reads another that has left
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

template <int V, bool LINES, bool BF16>
cudaError_t launch_small(const OrthSmallParams &p, cudaStream_t s) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(orth_small_kernel<V, LINES, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
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
    return cudaLaunchKernelEx(&cfg, orth_small_kernel<V, LINES, BF16>, p);
}

}  // namespace

cudaError_t launch_orth_small(const OrthSmallParams &p, cudaStream_t s) {
    const bool lines = rows_on_lines(p.bf16, {p.grad, p.result}, {p.momentum, p.weight}, p.copy, p.ld | p.ls | p.ldo | p.lse);
    if (p.cols % 4) return p.bf16 ? launch_small<1, false, true>(p, s) : launch_small<1, false, false>(p, s);
    if (lines) return p.bf16 ? launch_small<4, true, true>(p, s) : launch_small<4, true, false>(p, s);
    return p.bf16 ? launch_small<4, false, true>(p, s) : launch_small<4, false, false>(p, s);
}

}  // namespace cbd
