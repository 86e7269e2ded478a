/*
 * bsr_mx4.h -- microscaled 4-bit floating point: quantisation, expansion and the grouped product on
 * 4-bit weights (C ABI, same library and conventions as bsr_linear.h and bsr_experts.h).
 *
 * Memory-bound layers gain from weights that are loaded in a compact form and expanded on the GPU
 * (Lecture 11 summary, 48:12 "Load and Sparse Expand"), and sparsity composes with quantisation
 * (pytorch/ao sparsity README). The form is MXFP4 of the OCP Microscaling Formats specification:
 * 32 consecutive elements of a row share one scale byte, each element is an E2M1 code.
 *   code   4 bits: sign, then the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 for the low 3 bits 0 .. 7.
 *   byte   E8M0: the element's value is code * 2^(byte - 127); 255 is NaN.
 * Quantisation of a group with largest magnitude a > 0: byte = max(0, 127 + floor(log2 a) - 2), each
 * element divided by 2^(byte - 127) and rounded to the nearest magnitude, ties to the even code, above 6
 * to 6, sign kept. A group of zeros gets byte 0. A group that holds NaN or infinity gets byte 255 and
 * codes 0: all of it reads as NaN.
 *
 * Storage of a matrix of `rows` rows and K columns, K a multiple of 32 (contiguous, 16-byte aligned):
 *   codes  [rows][K/2] uint8, element 2i in the low half of byte i.
 *   scales [ceil(K/256)][rows][8] uint8: the 8 scale bytes of a row's 256 columns side by side, rows
 *          next to each other, so that a tile's scales are one contiguous piece. Bytes of groups at or
 *          past K are written 0 and never used.
 * Weights of E experts: codes [E][N][K/2], scales [E][ceil(K/256)][N][8].
 */
#ifndef BSR_MX4_H
#define BSR_MX4_H

#include <stddef.h>
#include <stdint.h>

#include "bsr_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Quantise X [rows][K] bf16 into codes and scales. values: NULL, or bf16 [rows][K] that receives what the
 * codes stand for (exact), in the same pass. rows >= 0, K a positive multiple of 32. Bit-exact. */
int32_t bsr_mx4_quantize(const bsr_bf16 *X, int64_t rows, int32_t K, uint8_t *codes, uint8_t *scales,
                         bsr_bf16 *values, void *stream);

/* Expand codes and scales to bf16: exact, and infinity for the values of bytes 253 and 254 that pass bf16's
 * range (quantisation gives byte 252 at most). */
int32_t bsr_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t K, bsr_bf16 *values,
                           void *stream);

/* bsr_expert_fwd with 4-bit weights: Y[r] = x(r) . W4[e]^T + bias[e], bf16 activations, fp32 sums.
 * codes [E][N][K/2], scales [E][ceil(K/256)][N][8]; K a multiple of 32, N of 8. The plain linear layer is
 * E = 1 with offsets {0, R}. X, gathered or sorted, at most 0xF0000000 bytes. */
int32_t bsr_expert_fwd_mx4(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                           const int32_t *offsets, const int32_t *row_token, const uint8_t *codes,
                           const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y, void *stream);

/* The same with both sides in 4 bits: x(r) is the row of xcodes [T or R][K/2] and
 * xscales [ceil(K/256)][T or R][8], xcodes at most 0xF0000000 bytes. Products of codes and scales are exact, sums are fp32. */
int32_t bsr_expert_fwd_mx4_mx4(const uint8_t *xcodes, const uint8_t *xscales, int64_t T, int64_t R, int32_t E,
                               int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_token,
                               const uint8_t *codes, const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y,
                               void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BSR_MX4_H */
