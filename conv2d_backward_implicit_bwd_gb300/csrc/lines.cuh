// lines.cuh -- bf16 rows at any address, read in whole 16-byte lines and shifted.
#pragma once
#include <stdint.h>

namespace cbd {

// The elements of a 16-byte line that lie in [begin, end), zeros elsewhere.  (Only at the ends of a tensor: short code.)
__device__ __forceinline__ uint4 line_by_element(uintptr_t line, uintptr_t begin, uintptr_t end) {
    uint64_t a = 0, b = 0;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const uintptr_t u = line + 2 * q, v = u + 8;
        if (u >= begin && u < end) a |= (uint64_t)*reinterpret_cast<const uint16_t *>(u) << (16 * q);
        if (v >= begin && v < end) b |= (uint64_t)*reinterpret_cast<const uint16_t *>(v) << (16 * q);
    }
    return make_uint4((uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32));
}
// eight elements from element s of lo on, over two lines
__device__ __forceinline__ uint4 shifted(const uint4 &lo, const uint4 &hi, int s) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = s & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = s & 2 ? w[i + 1] : w[i];
    const uint32_t by = (s & 1) * 16;
    return make_uint4(__funnelshift_r(w[0], w[1], by), __funnelshift_r(w[1], w[2], by), __funnelshift_r(w[2], w[3], by),
                      __funnelshift_r(w[3], w[4], by));
}

// a line of the tensor [begin, end): whole where it lies inside
__device__ __forceinline__ uint4 load_line(uintptr_t line, uintptr_t begin, uintptr_t end) {
    return line >= begin && line + 16 <= end ? *reinterpret_cast<const uint4 *>(line) : line_by_element(line, begin, end);
}

}  // namespace cbd
