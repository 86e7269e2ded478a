/*
 * bsr_expert_ffn.h -- a whole layer of experts for a few tokens (C ABI, same library and conventions as bsr_linear.h and
 * bsr_experts.h): router, top k, gate and up product, activation, down product and weighted sum in one call.
 *
 * The single calls of bsr_experts.h make a decode step of one layer some nine launches, whose starts cost more than a small
 * layer's weights take to read. Here each expert that some token chose is read once, for all tokens together.
 *   l[t]     = x[t] . router^T, fp32
 *   index[t] = the k experts of largest l, ties to the lowest expert; weight[t] their softmax weights, over all experts
 *              (renormalize = 0) or over the chosen ones (renormalize = 1); as bsr_router_fwd on l
 *   h[t][j]  = silu(g) * u with (g, u) = x[t] . up[e]^T + up_bias[e], e = index[t][j]; rounded to bf16 once
 *   out[t]   = sum over j of weight[t][j] * (h[t][j] . down[e]^T + down_bias[e]); fp32 sums, one rounding to bf16
 * A slot without an expert (logits of -infinity) adds nothing. Fixed order of sums: the result repeats bit for bit.
 */
#ifndef BSR_EXPERT_FFN_H
#define BSR_EXPERT_FFN_H

#include <stddef.h>
#include <stdint.h>

#include "bsr_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The most tokens of a call. */
#define BSR_EXPERT_FFN_TOKENS 16

/* How the weights of up and down are held. */
enum bsr_weight_form {
    BSR_WEIGHTS_BF16 = 0,   /* [E][rows][columns] bf16; scales NULL */
    BSR_WEIGHTS_MX4 = 1,    /* bsr_mx4.h: codes [E][rows][columns/2], scales [E][ceil(columns/256)][rows][8] */
    BSR_WEIGHTS_FP8 = 2     /* bsr_fp8_blocks.h: codes [E][rows][columns], scales [E][ceil(rows/128)][ceil(columns/128)],
                               which may start at any byte */
};

/* Bytes of device workspace that bsr_expert_ffn needs (0 for sizes that it refuses). */
size_t bsr_expert_ffn_workspace(int32_t T, int32_t dim, int32_t hidden, int32_t E, int32_t k);

/* out [T][dim] bf16 of x [T][dim] bf16, 0 <= T <= BSR_EXPERT_FFN_TOKENS.
 *   router    device bf16 [E][dim], 1 <= E <= 1024, 1 <= k <= min(32, E)
 *   form      bsr_weight_form, of both weights
 *   up        rows 2 * hidden (gate, then up), columns dim; up_bias bf16 [E][2 * hidden] or NULL
 *   down      rows dim, columns hidden; down_bias bf16 [E][dim] or NULL
 *   dim and hidden: positive multiples of 8 (bf16), 16 (fp8) or 32 (mx4), below 2^20 and 2^19; one expert's weight at most 0xF0000000
 *             bytes
 *   workspace device, 16-byte aligned, at least bsr_expert_ffn_workspace bytes; two calls that may run at the same time
 *             need one each. */
int32_t bsr_expert_ffn(const bsr_bf16 *x, int32_t T, int32_t dim, int32_t hidden, int32_t E, int32_t k,
                       int32_t renormalize, const bsr_bf16 *router, int32_t form, const void *up, const uint8_t *up_scales,
                       const void *down, const uint8_t *down_scales, const bsr_bf16 *up_bias, const bsr_bf16 *down_bias,
                       bsr_bf16 *out, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BSR_EXPERT_FFN_H */
