/*
 * bsr_fp8_blocks.h -- 8-bit floating point with a scale for each block of 128: quantisation, expansion and the
 * product grouped by expert (C ABI, same library and conventions as bsr_linear.h and bsr_experts.h).
 *
 * Dense weights and activations; bsr_fp8.h holds the blocks of a block-sparse weight in 8 bits. A compact form that is
 * expanded on the GPU serves layers that are bound by memory (Lecture 11 summary, 48:12 "Load and Sparse Expand"); on
 * activations as well it doubles the rate of the matrix cores.
 *   code   E4M3 of the OCP 8-bit floating point specification (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; exponent
 *          field 0 holds m * 2^-9; largest magnitude 448; 0x7F and 0xFF are NaN).
 *   byte   E8M0, as in bsr_mx4.h: the element's value is code * 2^(byte - 127); 255 is NaN.
 * Powers of two keep v / 2^s and code * 2^s exact, and the matrix instruction applies them by itself.
 * Quantisation of a group whose largest finite magnitude is a: s is the smallest integer >= -127 with a <= 448 * 2^s (-127
 * if a = 0), byte = s + 127 (at most 247), code = v / 2^s rounded to the nearest E4M3 value, ties to the even code, sign
 * kept. (Magnitudes above 248 * 2^120 become 256 * 2^120 = 2^128, which is past the range of bf16 and fp32.) NaN and the infinities become NaN codes of their sign (E4M3 has no infinity); the rest of the group is as without them.
 *
 * Storage (contiguous, 16-byte aligned; K a positive multiple of 16):
 *   rows    activations and gradients [rows][K]: a group is 128 columns of a row (the last one may be shorter).
 *           codes [rows][K]; scales [ceil(K/512)][rows][4], the bytes of a row's 512 columns side by side (those of groups
 *           at or past K are written 0 and never used).
 *   blocks  weights [E][N][K]: a group is 128 rows by 128 columns of one matrix, cut at its ends.
 *           codes [E][N][K]; scales [E][ceil(N/128)][ceil(K/128)]. Where they are read the scales may start at any byte, so that a slice
 *           of the experts serves as it is.
 */
#ifndef BSR_FP8_BLOCKS_H
#define BSR_FP8_BLOCKS_H

#include <stddef.h>
#include <stdint.h>

#include "bsr_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantise X [rows][K] bf16 by rows. values: NULL, or bf16 [rows][K] that receives what the codes stand for (exact), in the
 * same pass. rows >= 0. Bit-exact. */
int32_t bsr_fp8_quantize_rows(const bsr_bf16 *X, int64_t rows, int32_t K, uint8_t *codes, uint8_t *scales,
                              bsr_bf16 *values, void *stream);

/* Quantise W [E][N][K] bf16 by blocks. codes_t, scales_t: both NULL, or [E][K][N] and [E][ceil(K/128)][ceil(N/128)] that
 * receive the transposed matrices in the same form (a square group transposes into one), in the same pass.
 * E >= 1, N a positive multiple of 8 (of 16 with codes_t), below 2^20 each. Bit-exact. */
int32_t bsr_fp8_quantize_blocks(const bsr_bf16 *W, int32_t E, int32_t N, int32_t K, uint8_t *codes, uint8_t *scales,
                                uint8_t *codes_t, uint8_t *scales_t, void *stream);

/* Expand rows or blocks to bf16: exact wherever bf16 holds the value (every value below 2^128 that quantisation of bf16
 * gives), else rounded to the nearest, infinity past bf16's range. */
int32_t bsr_fp8_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t K, bsr_bf16 *values,
                                void *stream);
int32_t bsr_fp8_dequantize_blocks(const uint8_t *codes, const uint8_t *scales, int32_t E, int32_t N, int32_t K,
                                  bsr_bf16 *values, void *stream);

/* bsr_expert_fwd with 8-bit weights: Y[r] = x(r) . W8[e]^T + bias[e], bf16 activations, fp32 sums, one rounding.
 * codes [E][N][K], scales [E][ceil(N/128)][ceil(K/128)]; K a multiple of 16, N of 8. The plain linear layer is E = 1
 * with offsets {0, R}. X, gathered or sorted, at most 0xF0000000 bytes, and so is one expert's weight. Weights are expanded
 * to bf16 first: exact for what quantisation of bf16 gives. */
int32_t bsr_expert_fwd_fp8(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                           const int32_t *offsets, const int32_t *row_token, const uint8_t *codes,
                           const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y, void *stream);

/* The same with both sides in 8 bits: x(r) is the row of xcodes [T or R][K] and xscales [ceil(K/512)][T or R][4], xcodes at
 * most 0xF0000000 bytes. The matrix cores add the products of eight neighbouring columns (8 i to 8 i + 7) aligned to the
 * largest of their exponents and drop what lies below 2^-13 of it; everything beyond that is summed in fp32. (Expanded to bf16,
 * whose products lose nothing, the product would take twice the time.) The input gradient of a layer is this call on the
 * quantised dY [R][N] and the transposed weights. */
int32_t bsr_expert_fwd_fp8_fp8(const uint8_t *xcodes, const uint8_t *xscales, int64_t T, int64_t R, int32_t E,
                               int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_token,
                               const uint8_t *codes, const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BSR_FP8_BLOCKS_H */
