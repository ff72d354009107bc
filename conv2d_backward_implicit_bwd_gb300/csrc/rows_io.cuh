// rows_io.cuh -- V elements of a row at a time, fp32 or bf16: as one vector where addresses and strides allow it (LINES), else
// one by one.  V goes by the width alone, so that what is summed in the same order does not depend on where a tensor lies.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include <initializer_list>

namespace cbd {

template <int V, bool LINES, bool BF16>
__device__ __forceinline__ void load_v(const void *x, int64_t i, float (&v)[V]) {
    if constexpr (V == 1 || !LINES) {
#pragma unroll
        for (int l = 0; l < V; ++l) v[l] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i + l]) : static_cast<const float *>(x)[i + l];
    } else if constexpr (BF16) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(x) + i);
        v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u), v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
}
// (past L1: written by another thread of the block)
template <int V, bool LINES>
__device__ __forceinline__ void load_fresh(const float *x, float (&v)[V]) {
    if constexpr (V == 1 || !LINES) {
#pragma unroll
        for (int l = 0; l < V; ++l) v[l] = __ldcg(x + l);
    } else {
        const float4 f = __ldcg(reinterpret_cast<const float4 *>(x));
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    }
}
template <int V, bool LINES, bool BF16>
__device__ __forceinline__ void store_v(void *x, int64_t i, const float (&v)[V]) {
    if constexpr (V == 1 || !LINES) {
#pragma unroll
        for (int l = 0; l < V; ++l) {
            if constexpr (BF16)
                static_cast<__nv_bfloat16 *>(x)[i + l] = __float2bfloat16_rn(v[l]);
            else
                static_cast<float *>(x)[i + l] = v[l];
        }
    } else if constexpr (BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(x) + i) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(x) + i) = make_float4(v[0], v[1], v[2], v[3]);
    }
}
// Whether four elements are a vector everywhere: of the tensors in the input's type, of the fp32 ones, of a bf16 copy; the
// strides' bits.
inline bool rows_on_lines(bool bf16, std::initializer_list<const void *> typed, std::initializer_list<const void *> fp32, const void *copy, int64_t strides) {
    uintptr_t on16 = 0, on8 = reinterpret_cast<uintptr_t>(copy);
    for (const void *t : typed) (bf16 ? on8 : on16) |= reinterpret_cast<uintptr_t>(t);
    for (const void *t : fp32) on16 |= reinterpret_cast<uintptr_t>(t);
    return on16 % 16 == 0 && on8 % 8 == 0 && (strides & 3) == 0;
}

}  // namespace cbd
