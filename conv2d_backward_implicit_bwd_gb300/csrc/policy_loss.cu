// policy_loss.cu -- clipped policy loss with a KL term over logits rows:
// forward, backward, and both in one launch.
//
// Per row: m = max z, s = sum exp(scale (z - m)) in one pass (the running sum
// is rescaled when the maximum grows), logp = scale (z_a - m) - log s, the
// loss and its derivative c = dloss/dlogp from four floats, then
// dz_v = c scale ([v = a] - exp(scale (z_v - m)) / s) in a second pass.
// The fused form's second pass re-reads the row that this block has just read,
// from L2; memory sees each logit once and each gradient once.
#include <cuda_bf16.h>
#include <math.h>

#include "device_util.cuh"
#include "internal.h"
#include "train.h"

namespace cbd {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int NT = 256;
constexpr int UNR = 4;  // 16-byte loads of a thread in flight

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
};

// running maximum and sum of exp((z - m) c)
struct MaxSum {
    float m, s;
};
// Elements at -inf add 0 and leave the maximum; a NaN reaches s (fmaxf drops it from m).
template <int N>
__device__ __forceinline__ void take(MaxSum &r, const float (&v)[N], float c) {
    float m = r.m;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, v[i]);
    const float base = m == -INFINITY ? 0.f : m;
    float s = r.s * ex2((r.m - base) * c);
#pragma unroll
    for (int i = 0; i < N; ++i) s += ex2((v[i] - base) * c);
    r.m = m;
    r.s = s;
}
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float c) {
    MaxSum r;
    r.m = fmaxf(a.m, b.m);
    const float base = r.m == -INFINITY ? 0.f : r.m;
    r.s = a.s * ex2((a.m - base) * c) + b.s * ex2((b.m - base) * c);
    return r;
}

// Threads of one row: a whole block, or a warp (narrow vocabularies).
template <int TPR>
struct Group {
    static constexpr int ROWS = NT / TPR;
    static __device__ __forceinline__ int lane() { return threadIdx.x % TPR; }
    static __device__ __forceinline__ MaxSum reduce(MaxSum r, float c, MaxSum *sh) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            MaxSum o;
            o.m = __shfl_xor_sync(0xffffffffu, r.m, d);
            o.s = __shfl_xor_sync(0xffffffffu, r.s, d);
            r = merge(r, o, c);
        }
        if constexpr (TPR > 32) {
            if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = r;
            __syncthreads();
            r = sh[0];
#pragma unroll
            for (int w = 1; w < TPR / 32; ++w) r = merge(r, sh[w], c);
            __syncthreads();
        } else {
            __syncwarp();  // every lane has read its row: dlogits may overwrite it
        }
        return r;
    }
};

template <typename T, int TPR, int MODE>
__global__ void __launch_bounds__(NT) policy_kernel(const PolicyParams p) {
    using G = Group<TPR>;
    constexpr int VN = Vec<T>::N;
    __shared__ MaxSum sh[NT / 32];
    __shared__ double block_loss[G::ROWS];
    const int lane = G::lane(), sub = threadIdx.x / TPR;
    const int V = p.vocab;
    const float c = p.scale * kLog2e;
    double loss = 0.0;

    for (int64_t t = (int64_t)blockIdx.x * G::ROWS + sub; t < p.tokens; t += (int64_t)gridDim.x * G::ROWS) {
        const T *z = static_cast<const T *>(p.logits) + t * p.ld;
        T *dz = MODE == kPolForward ? nullptr : static_cast<T *>(p.dlogits) + t * p.ldd;
        const int a = p.actions[t];
        bool live;
        if constexpr (MODE == kPolBackward)
            live = a >= 0 && p.coef_in[t] != 0.f;
        else
            live = a >= 0 && p.weight[t] != 0.f;
        if (a >= V) {
            live = false;
            if (lane == 0) record_status(p.status, kDevFaultIndex);
        }
        // elements before the first 16-byte boundary, 16-byte vectors, the rest
        const int head = min(V, (int)((16 - ((uintptr_t)z & 15)) % 16 / sizeof(T)));
        const int nv = (V - head) / VN;
        const uint4 *zv = reinterpret_cast<const uint4 *>(z + head);

        float cs = 0.f, base = 0.f, inv = 0.f;  // dz = cs [v = a] - cs inv exp((z - base) c)
        if constexpr (MODE == kPolBackward) {
            if (live) {
                cs = p.coef_in[t] * (p.grad ? *p.grad : 1.f) * p.scale;
                base = p.lse_in[t];
            }
        } else if (live) {
            MaxSum r = {-INFINITY, 0.f};
            for (int i = lane; i < head; i += TPR) {
                const float v[1] = {Vec<T>::get(z + i)};
                take<1>(r, v, c);
            }
            int i = lane;
            for (; i + (UNR - 1) * TPR < nv; i += UNR * TPR) {
                uint4 u[UNR];
#pragma unroll
                for (int q = 0; q < UNR; ++q) u[q] = zv[i + q * TPR];
                float v[UNR * VN];
#pragma unroll
                for (int q = 0; q < UNR; ++q) {
                    float w[VN];
                    Vec<T>::unpack(u[q], w);
#pragma unroll
                    for (int k = 0; k < VN; ++k) v[q * VN + k] = w[k];
                }
                take<UNR * VN>(r, v, c);
            }
            for (; i < nv; i += TPR) {
                float w[VN];
                Vec<T>::unpack(zv[i], w);
                take<VN>(r, w, c);
            }
            for (int k = head + nv * VN + lane; k < V; k += TPR) {
                const float v[1] = {Vec<T>::get(z + k)};
                take<1>(r, v, c);
            }
            const float za = Vec<T>::get(z + a);
            r = G::reduce(r, c, sh);
            const float logs = logf(r.s);
            const float logp = (za - r.m) * p.scale + -logs;
            const float w = p.weight[t], adv = p.advantage[t];
            const float ratio = p.old_logp ? expf(logp - p.old_logp[t]) : 1.f;
            const float ra = ratio * adv, ca = fminf(fmaxf(ratio, p.clip_lo), p.clip_hi) * adv;
            const bool free_ = !(ra > ca);
            float l = -(free_ ? ra : ca), k = free_ ? -ra : 0.f;
            if (p.ref_logp && p.kl > 0.f) {
                const float d = p.ref_logp[t] - logp, ed = expm1f(d);
                l += p.kl * (ed - d);
                k -= p.kl * ed;
            }
            if (!p.old_logp && logp != logp) l = k = logp;  // no distribution: r = 1 would hide it
            if (lane == 0) {
                loss += (double)w * (double)l;
                p.logp[t] = logp;
                if (p.lse) p.lse[t] = r.m * p.scale + logs;
                if (p.coef) p.coef[t] = w * k;
            }
            cs = w * k * p.scale;
            base = r.m;
            inv = 1.f / r.s;
        } else if (lane == 0) {
            p.logp[t] = 0.f;
            if (p.lse) p.lse[t] = 0.f;
            if (p.coef) p.coef[t] = 0.f;
        }

        if constexpr (MODE != kPolForward) {
            auto grad_of = [&](float v, bool chosen) {
                float e;
                if constexpr (MODE == kPolBackward)
                    e = ex2((v * p.scale - base) * kLog2e);
                else
                    e = ex2((v - base) * c) * inv;
                return cs * ((chosen ? 1.f : 0.f) - e);
            };
            const bool same = (((uintptr_t)z ^ (uintptr_t)dz) & 15) == 0;
            const int dhead = live && !same ? V : min(V, (int)((16 - ((uintptr_t)dz & 15)) % 16 / sizeof(T)));
            const int dnv = (V - dhead) / VN;
            uint4 *dv = reinterpret_cast<uint4 *>(dz + dhead);
            if (!live) {
                for (int i = lane; i < dhead; i += TPR) Vec<T>::put(dz + i, 0.f);
                for (int i = lane; i < dnv; i += TPR) dv[i] = make_uint4(0u, 0u, 0u, 0u);
                for (int k = dhead + dnv * VN + lane; k < V; k += TPR) Vec<T>::put(dz + k, 0.f);
            } else {
                for (int i = lane; i < dhead; i += TPR) Vec<T>::put(dz + i, grad_of(Vec<T>::get(z + i), i == a));
                auto one = [&](int i, const uint4 &u) {
                    float w[VN], o[VN];
                    Vec<T>::unpack(u, w);
                    const int k0 = dhead + i * VN;
#pragma unroll
                    for (int k = 0; k < VN; ++k) o[k] = grad_of(w[k], k0 + k == a);
                    dv[i] = Vec<T>::pack(o);
                };
                int i = lane;
                for (; i + (UNR - 1) * TPR < dnv; i += UNR * TPR) {
                    uint4 u[UNR];
#pragma unroll
                    for (int q = 0; q < UNR; ++q) u[q] = zv[i + q * TPR];
#pragma unroll
                    for (int q = 0; q < UNR; ++q) one(i + q * TPR, u[q]);
                }
                for (; i < dnv; i += TPR) one(i, zv[i]);
                for (int k = dhead + dnv * VN + lane; k < V; k += TPR) Vec<T>::put(dz + k, grad_of(Vec<T>::get(z + k), k == a));
            }
        }
    }

    if constexpr (MODE != kPolBackward) {
        // the block's rows in order, then the blocks in order: a fixed sum
        if (lane == 0) block_loss[sub] = loss;
        __syncthreads();
        __shared__ bool last;
        if (threadIdx.x == 0) {
            double s = 0.0;
            for (int i = 0; i < G::ROWS; ++i) s += block_loss[i];
            p.partials[blockIdx.x] = s;
            __threadfence();
            last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
        }
        __syncthreads();
        if (last) {
            __threadfence();
            __shared__ double sums[NT];
            double s = 0.0;
            for (int i = threadIdx.x; i < (int)gridDim.x; i += NT) s += __ldcg(p.partials + i);
            sums[threadIdx.x] = s;
            __syncthreads();
            if (threadIdx.x < 32) {
                s = 0.0;
                for (int i = threadIdx.x; i < NT; i += 32) s += sums[i];
#pragma unroll
                for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                if (threadIdx.x == 0) {
                    *p.loss = (float)s;
                    *p.ticket = 0;
                }
            }
        }
    }
}

constexpr int kBlocksPerSm = 8;

template <typename T, int TPR>
cudaError_t launch_mode(const PolicyParams &p, int mode, int num_sms, cudaStream_t s) {
    const int64_t need = (p.tokens + NT / TPR - 1) / (NT / TPR);
    const int grid = (int)(need < 1 ? 1 : need < policy_max_blocks(num_sms) ? need : policy_max_blocks(num_sms));
    if (mode == kPolForward)
        policy_kernel<T, TPR, kPolForward><<<grid, NT, 0, s>>>(p);
    else if (mode == kPolBackward)
        policy_kernel<T, TPR, kPolBackward><<<grid, NT, 0, s>>>(p);
    else
        policy_kernel<T, TPR, kPolBoth><<<grid, NT, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

int policy_max_blocks(int num_sms) { return num_sms * kBlocksPerSm; }

cudaError_t launch_policy(const PolicyParams &p, int dtype, int mode, int num_sms, cudaStream_t s) {
    const bool narrow = p.vocab <= 1024;
    if (dtype == 1)
        return narrow ? launch_mode<__nv_bfloat16, 32>(p, mode, num_sms, s) : launch_mode<__nv_bfloat16, NT>(p, mode, num_sms, s);
    return narrow ? launch_mode<float, 32>(p, mode, num_sms, s) : launch_mode<float, NT>(p, mode, num_sms, s);
}

}  // namespace cbd
