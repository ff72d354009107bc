// vocab_rows.cuh -- rows of logits in 16-byte vectors, and the hardware's 2^x: what the kernels over a vocabulary share.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace cbd {

constexpr float kLog2e = 1.4426950408889634f;

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

// The terms 2^(z c - off) of a row, off = m c rounded, for a reference m.  One FMA
// for each exponential; off's rounding is the same for a row's every term and cancels.
// Past |m c| = 256 it would be more than 2^-17: there the difference z - m is taken
// first (and rest is what off lacks, where sums of both meet).
struct Exps {
    bool near;
    float base, off, rest, c;
    __device__ __forceinline__ Exps(float m, float c_) : c(c_) {
        const float mc = __fmul_rn(m, c_);
        near = fabsf(mc) < 256.f;
        base = near || m == -INFINITY ? 0.f : m;
        off = near ? mc : 0.f;
        rest = near ? fmaf(m, c_, -mc) : 0.f;
    }
    template <bool NEAR>
    __device__ __forceinline__ float at(float z) const {
        return ex2(NEAR ? fmaf(z, c, -off) : (z - base) * c);
    }
    __device__ __forceinline__ float at_any(float z) const { return near ? at<true>(z) : at<false>(z); }
    // the exponent that brings a sum over another reference m to this one's terms
    __device__ __forceinline__ float shift(float m, float m_here) const {
        if (m == -INFINITY || m == m_here) return 0.f;
        const Exps o(m, c);
        return near && o.near ? o.off - off : fmaf(m - m_here, c, rest - o.rest);
    }
    __device__ __forceinline__ float from(float m, float m_here) const { return m == -INFINITY || m == m_here ? 1.f : ex2(shift(m, m_here)); }
};

}  // namespace cbd
