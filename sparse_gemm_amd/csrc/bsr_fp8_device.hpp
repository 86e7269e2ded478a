// bsr_fp8_device.hpp -- device helpers of 8-bit floating point with a scale for each block of 128
// (include/bsr_fp8_blocks.h).
#pragma once

#include "bsr_mx4_device.hpp"

namespace bsr {
namespace dev {

constexpr int kFp8Group = 128;

typedef short i16x2 __attribute__((ext_vector_type(2)));

// The conversion instructions take the scale as mx4_scale_bits gives it: expansion is exact where bf16 holds the
// value, quantisation divides by the scale and rounds to the nearest code, ties to the even one. (Checked for every bf16 value,
// code and scale byte that the format gives.)

// Scale byte of a group whose largest finite magnitude has the bf16 bits `top` (without its sign): 448 is 1.75 * 2^8.
__device__ __forceinline__ int fp8_scale_byte(uint32_t top) {
    return max((int)(top >> 7) - 8 + ((top & 0x7F) > 0x60 ? 1 : 0), 0);
}

// Largest finite magnitude's bits among the two bf16 values of a word, and `top`.
__device__ __forceinline__ uint32_t fp8_top(uint32_t top, uint32_t w) {
    const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
    return max(top, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
}

// The codes of 4 bf16 values (two in each word).
__device__ __forceinline__ uint32_t fp8_quantize4(uint32_t w0, uint32_t w1, float scale) {
    i16x2 q = {0, 0};
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, bf16_pair(w0), scale, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, bf16_pair(w1), scale, true);
    uint32_t c = __builtin_bit_cast(uint32_t, q);
    const uint32_t v[4] = {w0 & 0xFFFFu, w0 >> 16, w1 & 0xFFFFu, w1 >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i)   // NaN and the infinities
        if ((v[i] & 0x7F80u) == 0x7F80u) c = (c & ~(0xFFu << (8 * i))) | ((0x7Fu | (v[i] >> 8 & 0x80u)) << (8 * i));
    return c;
}

// out[j] = byte j of a[0], a[1], a[2], a[3], lowest first.
__device__ __forceinline__ void transpose4(const uint32_t (&a)[4], uint32_t (&out)[4]) {
    const uint32_t t0 = __builtin_amdgcn_perm(a[1], a[0], 0x05010400), t1 = __builtin_amdgcn_perm(a[1], a[0], 0x07030602);
    const uint32_t t2 = __builtin_amdgcn_perm(a[3], a[2], 0x05010400), t3 = __builtin_amdgcn_perm(a[3], a[2], 0x07030602);
    out[0] = __builtin_amdgcn_perm(t2, t0, 0x05040100);
    out[1] = __builtin_amdgcn_perm(t2, t0, 0x07060302);
    out[2] = __builtin_amdgcn_perm(t3, t1, 0x05040100);
    out[3] = __builtin_amdgcn_perm(t3, t1, 0x07060302);
}

// The 8 values of 8 codes.
__device__ __forceinline__ bf16x8 fp8_expand8(uint2 codes, float scale) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

}  // namespace dev
}  // namespace bsr
