// bsr_experts_internal.hpp -- launchers of the expert-layer kernels (include/bsr_experts.h) and of the
// microscaled 4-bit kernels (include/bsr_mx4.h).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

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

// What a grouped product reads besides its operands. T: rows of the gathered matrix.
struct ExpertShape {
    int T, R, E, N, K;
    const int32_t *offsets, *row_token;
};

int32_t launch_expert_fwd(const ExpertShape &s, const uint16_t *X, const uint16_t *W, const uint16_t *bias, uint16_t *Y,
                          void *stream);
// A grid's threads are counted in 32 bits.
inline int32_t check_grid(int64_t blocks, int threads, const char *what) {
    if (blocks * threads > (int64_t)UINT32_MAX) return fail(BSR_ERR_INVALID_ARG, std::string(what) + ": too large for one launch");
    return BSR_OK;
}

// Which tile a grouped product takes. R rows of E experts are known on the host, the experts' shares are not: the rule
// takes equal groups and compares the tiles' estimated times, rounds of work-groups * (steps * time of a
// step + 2 us for a tile's start and end). The times are measured (a product of one expert whose tiles fill the card
// once or twice, 4096 x 4096 and 4096 -> 14336): `alone` with one work-group a CU, `shared` with `slots` of them on
// the card. Measured both sides of the rule, us (rows an expert: few-row tiles | 128 x 128):
//   forward 4096 -> 4096, E = 1     16: 8 | 34    64: 10 | 35    128: 15 | 35    256: 28 | 36    384: 40 | 36
//   forward 1024 -> 2048, E = 8     16: 9 | 13    32: 12 | 13    48: 13 | 13     64: 22 | 13
//   forward 4096 -> 14336, E = 8    16: 160 | 166   24: 203 | 196   32: 208 | 169
//   input gradient of 4096 -> 14336, E = 1   16: 38 | 108    128: 43 | 108    384: 114 | 109
//   4-bit forward 4096 -> 14336, E = 8       16: 58 | 103    24: 65 | 103     48: 100 | 113    64: 107 | 115    96: 159 | 125
struct TileKind {
    int id, rows, cols, step, slots;
    double alone, shared;
};

inline double tile_time(const TileKind &k, int64_t R, int64_t E, int64_t cols, int64_t C) {
    const double groups = (double)std::min(E, R), each = (double)R / groups;
    const double row_tiles = E == 1 ? std::ceil(each / k.rows) : groups * std::max(1.0, each / k.rows + 0.5);
    const double tiles = row_tiles * std::ceil((double)cols / k.cols), steps = std::ceil((double)C / k.step);
    const bool one = tiles <= 256;
    const double rounds = tiles / (one ? 256 : k.slots);
    return (rounds <= 2 ? std::ceil(rounds) : rounds) * (steps * (one ? k.alone : k.shared) + 2.0);
}

template <int n>
int best_tile(const TileKind (&kinds)[n], int64_t R, int64_t E, int64_t cols, int64_t C) {
    int best = 0;
    for (int i = 1; i < n; ++i)
        if (tile_time(kinds[i], R, E, cols, C) < tile_time(kinds[best], R, E, cols, C)) best = i;
    return kinds[best].id;
}

// ids 1, 2, 4: 16 * id-row tiles that stream the weights (bsr_experts_few.hip); 128, 256: the square tiles
constexpr TileKind kFwdTiles[] = {{1, 16, 32, 256, 512, 0.40, 0.62}, {2, 32, 32, 256, 256, 0.50, 0.50},
                                  {4, 64, 32, 256, 256, 0.80, 0.84}, {128, 128, 128, 64, 512, 0.52, 1.00},
                                  {256, 256, 256, 64, 256, 1.55, 1.55}};
constexpr TileKind kBwdInputTiles[] = {{1, 16, 64, 256, 256, 0.65, 0.65}, {2, 32, 64, 256, 256, 0.75, 0.75},
                                       {4, 64, 64, 256, 256, 1.05, 1.05}, {128, 128, 128, 64, 512, 0.50, 1.00},
                                       {256, 256, 256, 64, 256, 1.60, 1.60}};
constexpr TileKind kFwdMx4Tiles[] = {{1, 16, 64, 256, 512, 0.45, 0.75}, {2, 32, 64, 256, 512, 0.60, 0.90},
                                     {128, 128, 128, 64, 512, 0.56, 1.00}};

// Row tiles that R rows in E groups and the rows past the plan can need.
inline int64_t max_row_tiles(int64_t R, int64_t E, int64_t bm) { return (R + std::min(E + 1, R) * (bm - 1)) / bm; }

// Output columns of a few-row tile of 16 mt rows. Input gradient: 32 (half lines, two work-groups a CU) while tiles of 64 leave
// half of the 256 CUs without one: one row of 8 experts, 10744 -> 312: 23 us against 31, one expert, 4096 -> 4096: 10 against
// 12; where they do not, 4 rows of 64 experts, 1536 -> 2048: 92 against 80. (Where tiles of 32 rows would leave as many idle,
// tiles of 16 are estimated faster.)
inline int few_cols_bwd_input(int mt, int64_t R, int64_t E, int64_t cols) {
    return mt == 1 && max_row_tiles(R, E, 16) * ((cols + 63) / 64) <= 128 ? 32 : 64;
}
// 4-bit weights, up to 16 rows a tile: 32 while tiles of 64 leave CUs without one. One row, one expert: 4096 -> 4096 7.5 us
// against 9.6, 8192 -> 312 of 8 experts 11.4 against 15.6; where they do not, 4 rows of 32 experts, 2048 -> 1024: 11.0
// against 8.9.
inline int few_cols_mx4(int mt, int64_t R, int64_t E, int64_t cols) {
    return mt == 1 && max_row_tiles(R, E, 16) * ((cols + 63) / 64) <= 256 ? 32 : 64;
}

int32_t launch_expert_fwd_few(const ExpertShape &s, int mt, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                              uint16_t *Y, void *stream);
int32_t launch_expert_bwd_input_few(const ExpertShape &s, int mt, const uint16_t *dY, const uint16_t *W, uint16_t *dX,
                                    void *stream);
int32_t launch_expert_fwd_few_mx4(const ExpertShape &s, int mt, const uint16_t *X, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream);
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
