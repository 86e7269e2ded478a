// bsr_mx4_device.hpp -- device helpers of the microscaled 4-bit form (include/bsr_mx4.h).
#pragma once

#include "bsr_device.hpp"

namespace bsr {
namespace dev {

// 2^(byte - 127): an exponent field, except for byte 0 (2^-127 is subnormal) and 255 (NaN).
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
    if (byte == 0) return __uint_as_float(0x00400000u);
    if (byte == 255) return __builtin_nanf("");
    return __uint_as_float(byte << 23);
}

// Magnitude of the low 3 bits of a code: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
__device__ __forceinline__ float mx4_magnitude(uint32_t m) {
    return m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
}

// The 32 values of one group: element 2i in the low half of byte i.
__device__ __forceinline__ void mx4_expand(u32x4 codes, uint32_t byte, float *v) {
    const float scale = mx4_scale(byte);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const uint32_t c = codes[i >> 3] >> (4 * (i & 7));
        const float m = mx4_magnitude(c & 7u) * scale;
        v[i] = (c & 8u) ? -m : m;
    }
}

}  // namespace dev
}  // namespace bsr
