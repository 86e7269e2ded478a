// bsr_mx4_device.hpp -- device helpers of the microscaled 4-bit form (include/bsr_mx4.h).
#pragma once

#include "bsr_device.hpp"

namespace bsr {
namespace dev {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// The conversion instructions of gfx950 take the scale as a 32-bit float's exponent field: field b is
// 2^(b - 127) for b up to 254, 2^-127 for b = 0 as well, and NaN for b = 255. Expansion is exact; quantisation divides by
// the scale and rounds to the nearest magnitude, ties to the even code, and saturates (checked for every code,
// scale byte and bf16 value).
__device__ __forceinline__ float mx4_scale_bits(uint32_t byte) { return __uint_as_float(byte << 23); }

// The 8 values of 4 bytes of codes, element 2i in the low half of byte i.
__device__ __forceinline__ bf16x8 mx4_expand8(uint32_t codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ bf16x2 bf16_pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// The codes of 8 bf16 values (two in each word of x).
__device__ __forceinline__ uint32_t mx4_quantize8(u32x4 x, float scale) {
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(x[0]), scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(x[1]), scale, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(x[2]), scale, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(x[3]), scale, 3);
}

}  // namespace dev
}  // namespace bsr
