// grad_clip.cu -- global gradient norm over many tensors, and clipping.
//
// norm = sqrt(sum g^2), coef = min(1, max_norm / (norm + 1e-6)), out = g coef.
// The tensors are cut into chunks of 32 KB; a block takes chunks b, b + grid,
// ... in a fixed order and writes one fp64 partial; the block that finishes
// last adds the partials in order and writes norm and coef, so the result does
// not depend on scheduling.  A second launch scales, walking the chunks
// backwards: what the first read last is still in L2.
//
// A thread squares and sums its elements of a chunk (at most 64) in fp32 and
// adds that to fp64.  Where its fp32 sum is infinite, NaN or below the normal
// range of products (elements above 1.8e19 or all below 1e-15), it sums those
// elements again in fp64: the norm is right wherever it is a normal fp32
// number, at fp32 speed (fp64 adds are 1/64 of the rate).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>

#include "train.h"

namespace cbd {

namespace {

constexpr int NT = 256;

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 scaled(const uint4 &u, float c) {
        return make_uint4(__float_as_uint(__uint_as_float(u.x) * c), __float_as_uint(__uint_as_float(u.y) * c),
                          __float_as_uint(__uint_as_float(u.z) * c), __float_as_uint(__uint_as_float(u.w) * c));
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 scaled(const uint4 &u, float c) {
        float v[8];
        unpack(u, v);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i] * c, v[2 * i + 1] * c);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// (volatile: all of a chunk's loads are issued before the first is used)
__device__ __forceinline__ uint4 ld16(const uint4 *p) {
    uint4 u;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

// n elements from src: elements before the first 16-byte boundary, vectors, the rest
template <typename T>
struct Span {
    int head, nv, n;
    __device__ __forceinline__ Span(const void *base, int n_) : n(n_) {
        head = min(n_, (int)((16 - ((uintptr_t)base & 15)) % 16 / sizeof(T)));
        nv = (n_ - head) / Elem<T>::N;
    }
    __device__ __forceinline__ int tail() const { return head + nv * Elem<T>::N; }
};

template <typename T>
__device__ __forceinline__ double chunk_squares(const T *src, int n) {
    constexpr int VN = Elem<T>::N, MOST = kClipChunk / 16 / NT;
    const Span<T> sp(src, n);
    const uint4 *v = reinterpret_cast<const uint4 *>(src + sp.head);
    float s = 0.f;
    uint32_t any = 0;
    auto add = [&](float x) {
        s = fmaf(x, x, s);
        any |= __float_as_uint(x) << 1;
    };
    if ((int)threadIdx.x < sp.head) add(Elem<T>::get(src + threadIdx.x));
    if (sp.tail() + (int)threadIdx.x < n) add(Elem<T>::get(src + sp.tail() + threadIdx.x));
    uint4 u[MOST];
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
        const int i = threadIdx.x + q * NT;
        u[q] = make_uint4(0u, 0u, 0u, 0u);
        if (i < sp.nv) u[q] = ld16(v + i);
    }
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
        float w[VN];
        Elem<T>::unpack(u[q], w);
#pragma unroll
        for (int k = 0; k < VN; ++k) add(w[k]);
    }
    if (s >= 1e-30f && s <= 3e38f) return (double)s;
    if (any == 0) return 0.0;
    double d = 0.0;
    auto addd = [&](float x) { d = fma((double)x, (double)x, d); };
    if ((int)threadIdx.x < sp.head) addd(Elem<T>::get(src + threadIdx.x));
    if (sp.tail() + (int)threadIdx.x < n) addd(Elem<T>::get(src + sp.tail() + threadIdx.x));
#pragma unroll 1
    for (int q = 0; q < MOST; ++q) {
        const int i = threadIdx.x + q * NT;
        if (i >= sp.nv) break;
        float w[VN];
        Elem<T>::unpack(v[i], w);
#pragma unroll 1
        for (int k = 0; k < VN; ++k) addd(w[k]);
    }
    return d;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T *src, T *dst, int n, float c) {
    const Span<T> sp(src, n);
    if (((uintptr_t)src ^ (uintptr_t)dst) & 15) {
        for (int i = threadIdx.x; i < n; i += NT) Elem<T>::put(dst + i, Elem<T>::get(src + i) * c);
        return;
    }
    constexpr int MOST = kClipChunk / 16 / NT;
    const uint4 *v = reinterpret_cast<const uint4 *>(src + sp.head);
    uint4 *o = reinterpret_cast<uint4 *>(dst + sp.head);
    if ((int)threadIdx.x < sp.head) Elem<T>::put(dst + threadIdx.x, Elem<T>::get(src + threadIdx.x) * c);
    if (sp.tail() + (int)threadIdx.x < n)
        Elem<T>::put(dst + sp.tail() + threadIdx.x, Elem<T>::get(src + sp.tail() + threadIdx.x) * c);
    uint4 u[MOST];
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
        const int i = threadIdx.x + q * NT;
        if (i < sp.nv) u[q] = ld16(v + i);
    }
#pragma unroll
    for (int q = 0; q < MOST; ++q) {
        const int i = threadIdx.x + q * NT;
        if (i < sp.nv) o[i] = Elem<T>::scaled(u[q], c);
    }
}

__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) v += sh[w];
    __syncthreads();
    return v;
}

// The tensors' addresses travel as kernel parameters: nothing to copy or keep
// between calls, and a captured launch holds its own.
template <int N, bool OUT>
struct Pointers {
    const void *g[N];
    void *o[OUT ? N : 1];
};

template <int N>
__global__ void __launch_bounds__(NT) clip_norm_kernel(const __grid_constant__ ClipParams p, const __grid_constant__ Pointers<N, false> at) {
    __shared__ double sh[NT / 32];
    __shared__ bool last;
    double sum = 0.0;
    ClipChunk next = p.chunks[max(min((int)blockIdx.x, p.num_chunks - 1), 0)];
    for (int i = blockIdx.x; i < p.num_chunks; i += gridDim.x) {
        const ClipChunk ch = next;
        next = p.chunks[min(i + (int)gridDim.x, p.num_chunks - 1)];
        if (ch.bf16)
            sum += chunk_squares(static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start, ch.n);
        else
            sum += chunk_squares(static_cast<const float *>(at.g[ch.tensor]) + ch.start, ch.n);
    }
    sum = block_sum(sum, sh);
    if (threadIdx.x == 0) {
        p.partials[p.partial_base + blockIdx.x] = sum;
        __threadfence();
        last = p.partial_total > 0 && atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int i = threadIdx.x; i < p.partial_total; i += NT) sum += __ldcg(p.partials + i);
    sum = block_sum(sum, sh);
    if (threadIdx.x == 0) {
        const float norm = (float)sqrt(sum);
        *p.norm = norm;
        if (p.want_coef) {
            const float c = isinf(p.max_norm) && norm == norm ? 1.f : p.max_norm / (norm + 1e-6f);
            *p.coef = c > 1.f ? 1.f : c;  // keeps a NaN
        }
        *p.ticket = 0;
    }
}

template <int N>
__global__ void __launch_bounds__(NT) clip_scale_kernel(const __grid_constant__ ClipParams p, const __grid_constant__ Pointers<N, true> at) {
    const float c = *p.coef;
    ClipChunk next = p.chunks[max(p.num_chunks - 1 - (int)blockIdx.x, 0)];
    for (int i = p.num_chunks - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x) {
        const ClipChunk ch = next;
        next = p.chunks[max(i - (int)gridDim.x, 0)];
        if (c == 1.f && at.g[ch.tensor] == at.o[ch.tensor]) continue;  // in place and nothing to clip
        if (ch.bf16)
            chunk_scale(static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start,
                        static_cast<__nv_bfloat16 *>(at.o[ch.tensor]) + ch.start, ch.n, c);
        else
            chunk_scale(static_cast<const float *>(at.g[ch.tensor]) + ch.start,
                        static_cast<float *>(at.o[ch.tensor]) + ch.start, ch.n, c);
    }
}

constexpr int FEW = 64;  // a small table for few tensors: the parameters are copied at every launch

template <int N>
cudaError_t norm_with(const ClipParams &p, const void *const *g, int tensors, int grid, cudaStream_t s) {
    Pointers<N, false> at;
    memcpy(at.g, g, (size_t)tensors * sizeof(void *));
    clip_norm_kernel<N><<<grid, NT, 0, s>>>(p, at);
    return cudaGetLastError();
}
template <int N>
cudaError_t scale_with(const ClipParams &p, const void *const *g, void *const *o, int tensors, int grid, cudaStream_t s) {
    Pointers<N, true> at;
    memcpy(at.g, g, (size_t)tensors * sizeof(void *));
    memcpy(at.o, o, (size_t)tensors * sizeof(void *));
    clip_scale_kernel<N><<<grid, NT, 0, s>>>(p, at);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_clip_norm(const ClipParams &p, const void *const *g, int tensors, int grid, cudaStream_t s) {
    return tensors <= FEW ? norm_with<FEW>(p, g, tensors, grid, s) : norm_with<kClipPtrs>(p, g, tensors, grid, s);
}
cudaError_t launch_clip_scale(const ClipParams &p, const void *const *g, void *const *o, int tensors, int grid, cudaStream_t s) {
    return tensors <= FEW ? scale_with<FEW>(p, g, o, tensors, grid, s) : scale_with<kClipPtrs>(p, g, o, tensors, grid, s);
}

}  // namespace cbd
