// grad_clip.cu -- global gradient norm over many tensors, and clipping.
//
// norm = sqrt(sum g^2), coef = min(1, max_norm / (norm + 1e-6)), out = g coef.
// Bound by memory: the norm reads every gradient, the scaling reads and writes it.
//
// The tensors are cut into chunks of 32 KB.  Where every block of one cooperative
// launch can have one chunk (up to some 10 MB), the gradients stay in registers
// between the sum and the scaling and are read once: 48 tensors of 200 000 fp32 in
// 6 us instead of 10.  Larger sets take two launches.  The norm (7.0 TB/s) streams
// chunks b, b + grid, ... of a block through a ring of bulk copies; the scaling
// walks them backwards, as what the norm read last is still in L2, with loads and
// stores in registers, two blocks per SM (four: 682 against 665 us for 700 M
// gradients; through the ring with bulk stores 719).
//
// A block's partial sum is fp64; the block that finishes last adds the partials in
// order, so the result does not depend on scheduling.  A thread squares and sums
// its elements of a chunk (at most 66) in fp32.  Where that sum is infinite, NaN
// or so small that squares were lost (elements above 1.8e19 or all below 1e-15),
// it sums those elements again in fp64: the norm is right wherever it is a normal
// fp32 number, at fp32 speed (the fp64 rate is 1/64).
#include <cuda_bf16.h>
#include <math.h>
#include <string.h>
#include <type_traits>

#include "device_util.cuh"
#include "internal.h"
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

constexpr int EACH = kClipChunk / 16 / NT;  // vectors of a thread in a chunk

// The same elements of a thread's part (below) in fp64, read once more.
template <typename T>
__device__ __noinline__ double squares64(const T *src, int n) {
    const Span<T> sp(src, n);
    double d = 0.0;
    auto add = [&](int i) {
        const double x = (double)Elem<T>::get(src + i);
        d = fma(x, x, d);
    };
    if ((int)threadIdx.x < sp.head) add(threadIdx.x);
    if (sp.tail() + (int)threadIdx.x < n) add(sp.tail() + threadIdx.x);
    for (int v = threadIdx.x; v < sp.nv; v += NT)
        for (int k = 0; k < Elem<T>::N; ++k) add(sp.head + v * Elem<T>::N + k);
    return d;
}

// A thread's part of a chunk, in registers: vectors, and at most one element
// before and one after them.
template <typename T>
struct Part {
    Span<T> sp;
    uint4 u[EACH];
    float head, tail;
    __device__ __forceinline__ Part(const T *src, int n) : sp(src, n), head(0.f), tail(0.f) {
        const uint4 *v = reinterpret_cast<const uint4 *>(src + sp.head);
#pragma unroll
        for (int q = 0; q < EACH; ++q) {
            u[q] = make_uint4(0u, 0u, 0u, 0u);
            if ((int)threadIdx.x + q * NT < sp.nv) u[q] = ld16(v + threadIdx.x + q * NT);
        }
        if ((int)threadIdx.x < sp.head) head = Elem<T>::get(src + threadIdx.x);
        if (sp.tail() + (int)threadIdx.x < n) tail = Elem<T>::get(src + sp.tail() + threadIdx.x);
    }
    __device__ __forceinline__ double squares(const T *src, int n) const {
        constexpr int VN = Elem<T>::N;
        float s = fmaf(head, head, tail * tail);
        uint32_t any = (__float_as_uint(head) | __float_as_uint(tail)) << 1;
#pragma unroll
        for (int q = 0; q < EACH; ++q) {
            float w[VN];
            Elem<T>::unpack(u[q], w);
#pragma unroll
            for (int k = 0; k < VN; ++k) s = fmaf(w[k], w[k], s);
            any |= u[q].x | u[q].y | u[q].z | u[q].w;
        }
        if (s >= 1e-30f && s <= 3e38f) return (double)s;
        if (any == 0) return 0.0;
        return squares64<T>(src, n);
    }
    __device__ __forceinline__ void store(T *dst, int n, float c) const {
        if ((int)threadIdx.x < sp.head) Elem<T>::put(dst + threadIdx.x, head * c);
        if (sp.tail() + (int)threadIdx.x < n) Elem<T>::put(dst + sp.tail() + threadIdx.x, tail * c);
        T *to = dst + sp.head;
        if (((uintptr_t)to & 15) == 0) {
            uint4 *o = reinterpret_cast<uint4 *>(to);
#pragma unroll
            for (int q = 0; q < EACH; ++q)
                if ((int)threadIdx.x + q * NT < sp.nv) o[threadIdx.x + q * NT] = Elem<T>::scaled(u[q], c);
        } else {
#pragma unroll
            for (int q = 0; q < EACH; ++q) {
                const int i = threadIdx.x + q * NT;
                if (i >= sp.nv) break;
                float w[Elem<T>::N];
                Elem<T>::unpack(u[q], w);
#pragma unroll
                for (int k = 0; k < Elem<T>::N; ++k) Elem<T>::put(to + i * Elem<T>::N + k, w[k] * c);
            }
        }
    }
};

// (threads past NT are there for the barriers and have nothing)
__device__ __forceinline__ double block_sum(double v, double *sh) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threadIdx.x % 32 == 0 && threadIdx.x < NT) sh[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) v += sh[w];
    __syncthreads();
    return v;
}

// By the block that finishes last: the partials in order, norm and coef.
__device__ __forceinline__ float finish(const ClipParams &p, int partials, double *sh) {
    double sum = 0.0;
    if (threadIdx.x < NT)
        for (int i = threadIdx.x; i < partials; i += NT) sum += __ldcg(p.partials + i);
    sum = block_sum(sum, sh);
    const float norm = (float)sqrt(sum);
    float c = isinf(p.max_norm) && norm == norm ? 1.f : p.max_norm / (norm + 1e-6f);
    c = c > 1.f ? 1.f : c;  // keeps a NaN
    if (threadIdx.x == 0) {
        *p.norm = norm;
        if (p.want_coef) *p.coef = c;
        *p.ticket = 0;
    }
    return c;
}

// The tensors' addresses travel as kernel parameters: nothing to copy or keep
// between calls, and a captured launch holds its own.
template <int N, bool OUT>
struct Pointers {
    const void *g[N];
    void *o[OUT ? N : 1];
};

// Chunks stream through a ring of half chunks in shared memory that one thread
// fills with bulk copies, three blocks per SM: 192 KB of reads stay in flight
// under the arithmetic (loads into registers, all of a chunk's at once, reached
// 4.4 TB/s).  Elements before a tensor's first 16-byte boundary and after the last
// are read directly.
constexpr int SLOT = kClipChunk / 2, RING = 4, NORM_BLOCKS = kNormBlocks;
constexpr int kNormSmem = SLOT * RING + 2 * RING * 8;

template <typename T>
__device__ __forceinline__ int slots_of(const T *src, int n) {
    return (Span<T>(src, n).nv * 16 + SLOT - 1) / SLOT;
}

template <int N>
__global__ void __launch_bounds__(NT + 32, NORM_BLOCKS) clip_norm_kernel(const __grid_constant__ ClipParams p, const __grid_constant__ Pointers<N, false> at) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ double sh[NT / 32];
    __shared__ bool last;
    __shared__ int abort_;
    volatile int32_t *abort_flag = &abort_;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + SLOT * RING);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + RING);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(full0 + 8 * i, 1);
            mbar_init(empty0 + 8 * i, NT / 32);
        }
        abort_ = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    __syncthreads();
    uint32_t it = 0;
    bool ok = true;
    double sum = 0.0;
    ClipChunk next = p.chunks[max(min((int)blockIdx.x, p.num_chunks - 1), 0)];
    if (warp == NT / 32) {
        if (lane == 0) {
            for (int i = blockIdx.x; i < p.num_chunks && ok; i += gridDim.x) {
                const ClipChunk ch = next;
                next = p.chunks[min(i + (int)gridDim.x, p.num_chunks - 1)];
                const char *src;
                int bytes;
                if (ch.bf16) {
                    const __nv_bfloat16 *g = static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start;
                    const Span<__nv_bfloat16> sp(g, ch.n);
                    src = reinterpret_cast<const char *>(g + sp.head);
                    bytes = sp.nv * 16;
                } else {
                    const float *g = static_cast<const float *>(at.g[ch.tensor]) + ch.start;
                    const Span<float> sp(g, ch.n);
                    src = reinterpret_cast<const char *>(g + sp.head);
                    bytes = sp.nv * 16;
                }
                for (int o = 0; o < bytes; o += SLOT, ++it) {
                    const uint32_t b = it % RING, ph = (it / RING) & 1;
                    ok = mbar_wait_bounded(empty0 + 8 * b, ph ^ 1, p.wait_budget, abort_flag, p.status, kDevTimeoutProducer);
                    if (!ok) break;
                    const int size = min(SLOT, bytes - o);
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full0 + 8 * b), "r"(size) : "memory");
                    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(ring) + b * SLOT),
                                 "l"(src + o), "r"(size), "r"(full0 + 8 * b)
                                 : "memory");
                }
            }
            if (!ok) {
                for (int q = 0; q < 100; ++q) __nanosleep(1000);
            }
        }
        __syncwarp();
    } else {
        auto chunk = [&](const auto *src, int n) {
            using T = typename std::remove_cv<typename std::remove_pointer<decltype(src)>::type>::type;
            constexpr int VN = Elem<T>::N;
            const Span<T> sp(src, n);
            float s = 0.f;
            uint32_t any = 0;
            if ((int)threadIdx.x < sp.head) {
                const float x = Elem<T>::get(src + threadIdx.x);
                s = x * x;
                any = __float_as_uint(x) << 1;
            }
            if (sp.tail() + (int)threadIdx.x < n) {
                const float x = Elem<T>::get(src + sp.tail() + threadIdx.x);
                s = fmaf(x, x, s);
                any |= __float_as_uint(x) << 1;
            }
            const int slots = slots_of(src, n);
            for (int k = 0; k < slots; ++k, ++it) {
                if (ok) ok = mbar_wait_bounded(full0 + 8 * (it % RING), (it / RING) & 1, p.wait_budget, abort_flag, p.status, kDevTimeoutEpilogue);
                const uint4 *buf = reinterpret_cast<const uint4 *>(ring + (it % RING) * SLOT);
                const int m = min(SLOT / 16, sp.nv - k * (SLOT / 16));
#pragma unroll
                for (int q = 0; q < SLOT / 16 / NT; ++q) {
                    const int v = threadIdx.x + q * NT;
                    if (v >= m) break;
                    const uint4 u = buf[v];
                    float w[VN];
                    Elem<T>::unpack(u, w);
#pragma unroll
                    for (int j = 0; j < VN; ++j) s = fmaf(w[j], w[j], s);
                    any |= u.x | u.y | u.z | u.w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty0 + 8 * (it % RING));
            }
            sum += s >= 1e-30f && s <= 3e38f ? (double)s : any == 0 ? 0.0 : squares64<T>(src, n);
        };
        for (int i = blockIdx.x; i < p.num_chunks; i += gridDim.x) {
            const ClipChunk ch = next;
            next = p.chunks[min(i + (int)gridDim.x, p.num_chunks - 1)];
            if (ch.bf16)
                chunk(static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start, ch.n);
            else
                chunk(static_cast<const float *>(at.g[ch.tensor]) + ch.start, ch.n);
        }
        if (!ok) sum = nan("");  // a wait ran out: no norm
    }
    __syncthreads();
    sum = block_sum(sum, sh);
    if (threadIdx.x == 0) {
        p.partials[p.partial_base + blockIdx.x] = sum;
        __threadfence();
        last = p.partial_total > 0 && atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    finish(p, p.partial_total, sh);
}

template <int N>
__global__ void __launch_bounds__(NT) clip_scale_kernel(const __grid_constant__ ClipParams p, const __grid_constant__ Pointers<N, true> at) {
    const float c = *p.coef;
    ClipChunk next = p.chunks[max(p.num_chunks - 1 - (int)blockIdx.x, 0)];
    for (int i = p.num_chunks - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x) {
        const ClipChunk ch = next;
        next = p.chunks[max(i - (int)gridDim.x, 0)];
        if (c == 1.f && at.g[ch.tensor] == at.o[ch.tensor]) continue;  // in place and nothing to clip
        if (ch.bf16) {
            const Part<__nv_bfloat16> part(static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start, ch.n);
            part.store(static_cast<__nv_bfloat16 *>(at.o[ch.tensor]) + ch.start, ch.n, c);
        } else {
            const Part<float> part(static_cast<const float *>(at.g[ch.tensor]) + ch.start, ch.n);
            part.store(static_cast<float *>(at.o[ch.tensor]) + ch.start, ch.n, c);
        }
    }
}

// Few enough chunks for every block to have one, all resident (a cooperative
// launch): the gradients stay in registers from the sum to the scaling, read
// once.  The block that arrives last writes norm and coef and moves the turn on;
// the others wait for that (bounded: after a wait that ran out a block leaves its
// chunk as it is and the status says so).
template <typename T>
__device__ __forceinline__ void clip_one(const ClipParams &p, const T *src, T *dst, int n, double *sh, int *flag) {
    const uint32_t turn = *(volatile uint32_t *)p.turn;  // before this block arrives, so before it can move
    const Part<T> part(src, n);
    const double sum = block_sum(part.squares(src, n), sh);
    if (threadIdx.x == 0) {
        p.partials[blockIdx.x] = sum;
        __threadfence();
        *flag = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    const bool last = *flag;
    __syncthreads();  // the flag is written again
    float c = 1.f;
    if (last) {
        __threadfence();
        c = finish(p, gridDim.x, sh);
        if (threadIdx.x == 0) {
            __threadfence();
            asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p.turn), "r"(turn + 1) : "memory");
        }
    } else {
        if (threadIdx.x == 0) {
            const long long t0 = clock64();
            uint32_t now = turn;
            int ok = 1;
            while (now == turn) {
                asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(now) : "l"(p.turn) : "memory");
                if (now == turn && clock64() - t0 > p.wait_budget) {
                    record_status(p.status, kDevTimeoutPartial);
                    ok = 0;
                    break;
                }
            }
            *flag = ok;
            sh[0] = ok ? (double)__ldcg(p.coef) : 1.0;
        }
        __syncthreads();
        if (!*flag) return;
        c = (float)sh[0];
    }
    if (c == 1.f && src == dst) return;
    part.store(dst, n, c);
}

template <int N>
__global__ void __launch_bounds__(NT) clip_fused_kernel(const __grid_constant__ ClipParams p, const __grid_constant__ Pointers<N, true> at) {
    __shared__ double sh[NT / 32];
    __shared__ int flag;
    const ClipChunk ch = p.chunks[blockIdx.x];
    if (ch.bf16)
        clip_one(p, static_cast<const __nv_bfloat16 *>(at.g[ch.tensor]) + ch.start, static_cast<__nv_bfloat16 *>(at.o[ch.tensor]) + ch.start, ch.n, sh, &flag);
    else
        clip_one(p, static_cast<const float *>(at.g[ch.tensor]) + ch.start, static_cast<float *>(at.o[ch.tensor]) + ch.start, ch.n, sh, &flag);
}

constexpr int FEW = 64;  // a small table for few tensors: the parameters are copied at every launch

template <int N>
cudaError_t norm_with(const ClipParams &p, const void *const *g, int tensors, int grid, cudaStream_t s) {
    Pointers<N, false> at;
    memcpy(at.g, g, (size_t)tensors * sizeof(void *));
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(clip_norm_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    return launch_early(clip_norm_kernel<N>, grid, NT + 32, kNormSmem, s, p, at);
}
template <int N>
cudaError_t scale_with(const ClipParams &p, const void *const *g, void *const *o, int tensors, int grid, cudaStream_t s) {
    Pointers<N, true> at;
    memcpy(at.g, g, (size_t)tensors * sizeof(void *));
    memcpy(at.o, o, (size_t)tensors * sizeof(void *));
    // (not early: blocks that settle while the norm's leave would spread unevenly over the SMs, 827 against 637 us)
    clip_scale_kernel<N><<<grid, NT, 0, s>>>(p, at);
    return cudaGetLastError();
}

template <int N>
cudaError_t fused_with(const ClipParams &p, const void *const *g, void *const *o, int tensors, cudaStream_t s) {
    Pointers<N, true> at;
    memcpy(at.g, g, (size_t)tensors * sizeof(void *));
    memcpy(at.o, o, (size_t)tensors * sizeof(void *));
    void *args[] = {const_cast<ClipParams *>(&p), &at};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void *>(clip_fused_kernel<N>), dim3((unsigned)p.num_chunks), dim3(NT), args, 0, s);
}

}  // namespace

cudaError_t launch_clip_norm(const ClipParams &p, const void *const *g, int tensors, int grid, cudaStream_t s) {
    return tensors <= FEW ? norm_with<FEW>(p, g, tensors, grid, s) : norm_with<kClipPtrs>(p, g, tensors, grid, s);
}
cudaError_t launch_clip_scale(const ClipParams &p, const void *const *g, void *const *o, int tensors, int grid, cudaStream_t s) {
    return tensors <= FEW ? scale_with<FEW>(p, g, o, tensors, grid, s) : scale_with<kClipPtrs>(p, g, o, tensors, grid, s);
}

int clip_fused_blocks(int num_sms) {
    int few = 0, many = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&few, clip_fused_kernel<FEW>, NT, 0) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&many, clip_fused_kernel<kClipPtrs>, NT, 0) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return (few < many ? few : many) * num_sms;
}
cudaError_t launch_clip_fused(const ClipParams &p, const void *const *g, void *const *o, int tensors, cudaStream_t s) {
    return tensors <= FEW ? fused_with<FEW>(p, g, o, tensors, s) : fused_with<kClipPtrs>(p, g, o, tensors, s);
}

}  // namespace cbd
