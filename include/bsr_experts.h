/*
 * bsr_experts.h -- layers of experts: a router, products grouped by expert with ragged sizes, and
 * the sum over a token's experts (C ABI, same library and conventions as bsr_linear.h: raw bf16
 * bits, caller-owned contiguous device buffers aligned to 16 bytes, a hipStream_t passed as void*,
 * arguments checked before anything is enqueued, a bsr_status returned, no C++ exception across
 * the interface, nothing synchronised).
 *
 * A block-sparse layer keeps some blocks of one weight for every token (pytorch_block_sparse
 * summary page, "Block-Sparse Implementation and Usage"); a layer of experts keeps, for each token,
 * k of E dense weights. Seen over all tokens its weight is block sparse too, with one block column
 * per expert and a pattern that the router chooses anew in every step, so the pattern is an array
 * on the device and no call needs it on the host.
 *
 * Notation: T tokens, k slots a token, E experts (1 <= E <= 1024, 1 <= k <= 32, k <= E), R = T * k.
 *   index[T][k]     int32  expert of each slot; outside [0, E): the slot is dropped
 *   offsets[E+1]    int32  rows offsets[e] .. offsets[e+1] - 1 belong to expert e
 *   row_token[R]    int32  token of each row; -1 for rows at or past offsets[E]
 *   slot_row[T][k]  int32  row of each slot; -1 for dropped slots
 * Rows are ordered by expert, and by slot (t * k + j) inside an expert.
 *
 * The kernels clamp what they read from offsets to [0, R] and drop tokens and rows out of range, so
 * a plan that does not hold these invariants gives wrong results but no access out of bounds.
 * Size limits (BSR_ERR_INVALID_ARG beyond them): R <= 2^24; at most 0xF0000000 bytes for one expert's weight, for an X
 * whose rows are gathered by token, and for X and dY of the weight gradient; N and K below 2^20 and multiples of 8 (rows
 * of 16-byte pieces); less than 2^32 threads a launch. Sorted rows (X of the forward without row_token, dY of the input
 * gradient), results, and all experts' weights together may be of any size.
 */
#ifndef BSR_EXPERTS_H
#define BSR_EXPERTS_H

#include <stddef.h>
#include <stdint.h>

#include "bsr_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Type of the router's logits. */
enum bsr_logits_type { BSR_LOGITS_F32 = 0, BSR_LOGITS_BF16 = 1 };

/* Router: index[t] = the k largest of logits[t][0..E), largest first, ties to the lowest expert;
 * weight[t][j] = exp(l_j - m) / sum of exp(l_e - m), over all experts (renormalize = 0) or over the
 * k chosen ones (renormalize = 1); 32-bit arithmetic. A logit of -infinity is an expert that the
 * token may not use: a slot that finds nothing else gets index -1 and weight 0, so a row of -infinity
 * has no expert at all. NaN counts as the largest value and makes the row's weights NaN, as +infinity does.
 *   logits device [T][E] f32 or bf16 (type); index device [T][k] int32; weight device [T][k] f32. */
int32_t bsr_router_fwd(const void *logits, int32_t type, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                       int32_t *index, float *weight, void *stream);

/* Gradient of the router's weights: dlogits[t][E] of the logits' type from dweight[T][k] (f32), with
 * index and weight as bsr_router_fwd wrote them. The choice itself has no gradient.
 *   renormalize = 0: dl_e = p_e (g_e - sum_j w_j g_j), g_e = dweight of e's slot or 0
 *   renormalize = 1: dl_e = w_j (g_j - sum_i w_i g_i) for the chosen experts, 0 for the others */
int32_t bsr_router_bwd(const void *logits, int32_t type, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                       const int32_t *index, const float *weight, const float *dweight, void *dlogits, void *stream);

/* Up to so many slots (T * k) bsr_expert_plan needs no workspace. */
#define BSR_EXPERT_PLAN_SLOTS 1024

/* Bytes of device workspace that bsr_expert_plan needs (0 up to BSR_EXPERT_PLAN_SLOTS slots). */
size_t bsr_expert_plan_workspace(int64_t T, int32_t k, int32_t E);

/* The plan of an index: offsets, row_token and slot_row as above, by a stable counting sort on the
 * device (no atomics on the results' order: the same index gives the same plan).
 *   workspace device, 4-byte aligned, at least bsr_expert_plan_workspace(T, k, E) bytes. */
int32_t bsr_expert_plan(const int32_t *index, int64_t T, int32_t k, int32_t E, int32_t *offsets, int32_t *row_token,
                        int32_t *slot_row, void *workspace, size_t ws_bytes, void *stream);

/* Grouped forward: Y[r] = x(r) . W[e]^T + bias[e] for the rows r of each expert e.
 *   X         device bf16. With row_token: [T][K], x(r) = X[row_token[r]]. With row_token NULL:
 *             [R][K], x(r) = X[r] (T is not used).
 *   offsets   device [E+1] int32 of a plan with R rows.
 *   W         device [E][N][K] bf16; bias device [E][N] bf16 or NULL.
 *   Y         device [R][N] bf16; every row is written, rows at or past offsets[E] with 0. */
int32_t bsr_expert_fwd(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                       const int32_t *offsets, const int32_t *row_token, const bsr_bf16 *W, const bsr_bf16 *bias,
                       bsr_bf16 *Y, void *stream);

/* Grouped input gradient: dX[r] = dY[r] . W[e] for the rows r of each expert e; dX [R][K] bf16, rows at
 * or past offsets[E] are 0. (The gradient of a gathered X is the sum over a token's rows:
 * bsr_expert_combine_fwd with weight NULL.) */
int32_t bsr_expert_bwd_input(const bsr_bf16 *dY, int64_t R, int32_t E, int32_t N, int32_t K, const int32_t *offsets,
                             const bsr_bf16 *W, bsr_bf16 *dX, void *stream);

/* Grouped weight gradient: dW[e] = sum over the rows r of e of dY[r]^T . x(r), dbias[e] = sum of dY[r]
 * (either NULL to skip it, not both). X, T and row_token as for the forward. dW [E][N][K] bf16, dbias [E][N] bf16; experts
 * without rows get 0. Sums in fp32, in a fixed order: the result is deterministic. */
int32_t bsr_expert_bwd_weight(const bsr_bf16 *dY, const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N,
                              int32_t K, const int32_t *offsets, const int32_t *row_token, bsr_bf16 *dW,
                              bsr_bf16 *dbias, void *stream);

/* Sum over a token's rows: out[t] = sum over j of weight[t][j] * Y[slot_row[t][j]], dropped slots left
 * out; fp32 sums in slot order, one rounding. weight NULL: every weight 1.
 *   Y device [R][N] bf16; slot_row device [T][k] int32; weight device [T][k] f32; out device [T][N] bf16. */
int32_t bsr_expert_combine_fwd(const bsr_bf16 *Y, int64_t T, int32_t k, int32_t N, const int32_t *slot_row,
                               const float *weight, bsr_bf16 *out, void *stream);

/* Gradient of the sum: dY[slot_row[t][j]] = weight[t][j] * dout[t] (rows at or past offsets[E] are 0) and
 * dweight[t][j] = <dout[t], Y[slot_row[t][j]]> in fp32 (0 for dropped slots). */
int32_t bsr_expert_combine_bwd(const bsr_bf16 *dout, const bsr_bf16 *Y, int64_t T, int32_t k, int32_t E, int32_t N,
                               const int32_t *offsets, const int32_t *slot_row, const float *weight, bsr_bf16 *dY,
                               float *dweight, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* BSR_EXPERTS_H */
