// bsr_experts_internal.hpp -- launchers of the expert-layer kernels (include/bsr_experts.h) and of the
// microscaled 4-bit kernels (include/bsr_mx4.h).
#pragma once

#include <cstdint>

#include "bsr_experts.h"
#include "bsr_internal.hpp"
#include "bsr_mx4.h"

namespace bsr {

constexpr int kMaxExperts = 1024;
constexpr int kMaxSlots = 32;
constexpr int64_t kMaxExpertRows = 1 << 24;
constexpr uint64_t kMaxOperandBytes = 0xF0000000u;   // one matrix behind a buffer resource; offsets past it read zeros

int32_t launch_router_fwd(const void *logits, int32_t type, int T, int E, int k, bool renorm, int32_t *index,
                          float *weight, void *stream);
int32_t launch_router_bwd(const void *logits, int32_t type, int T, int E, int k, bool renorm, const int32_t *index,
                          const float *weight, const float *dweight, void *dlogits, void *stream);
size_t expert_plan_workspace_bytes(int64_t slots, int E);
int32_t launch_expert_plan(const int32_t *index, int T, int k, int E, int32_t *offsets, int32_t *row_token,
                           int32_t *slot_row, void *workspace, void *stream);
int32_t launch_combine_fwd(const uint16_t *Y, int T, int k, int N, const int32_t *slot_row, const float *weight,
                           uint16_t *out, void *stream);
int32_t launch_combine_bwd(const uint16_t *dout, const uint16_t *Y, int T, int k, int E, int N, const int32_t *offsets,
                           const int32_t *slot_row, const float *weight, uint16_t *dY, float *dweight, void *stream);

// What a grouped product reads besides its operands. rows_a: rows of the gathered matrix (T) or R.
struct ExpertShape {
    int T, R, E, N, K;
    const int32_t *offsets, *row_token;
};

int32_t launch_expert_fwd(const ExpertShape &s, const uint16_t *X, const uint16_t *W, const uint16_t *bias, uint16_t *Y,
                          void *stream);
// Few rows an expert: 16-row tiles that stream the weights.
inline bool few_rows(int64_t R, int64_t E) { return R <= 24 * E; }
int32_t launch_expert_fwd_few(const ExpertShape &s, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                              uint16_t *Y, void *stream);
int32_t launch_expert_fwd_few_mx4(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                                  const uint16_t *bias, uint16_t *Y, void *stream);
int32_t launch_expert_bwd_input(const ExpertShape &s, const uint16_t *dY, const uint16_t *W, uint16_t *dX, void *stream);
int32_t launch_expert_bwd_weight(const ExpertShape &s, const uint16_t *dY, const uint16_t *X, uint16_t *dW,
                                 uint16_t *dbias, void *stream);

int32_t launch_mx4_quantize(const uint16_t *X, int64_t rows, int K, uint8_t *codes, uint8_t *scales, uint16_t *values,
                            void *stream);
int32_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint16_t *values,
                              void *stream);
int32_t launch_expert_fwd_mx4(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream);
int32_t launch_expert_fwd_mx4_mx4(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales,
                                  const uint8_t *codes, const uint8_t *scales, const uint16_t *bias, uint16_t *Y,
                                  void *stream);

}  // namespace bsr
