// bsr_experts_internal.hpp -- launchers of the expert-layer kernels (include/bsr_experts.h) and of the
// microscaled 4-bit kernels (include/bsr_mx4.h), of the 8-bit ones (include/bsr_fp8_blocks.h) and of the whole layer for a few
// tokens (include/bsr_expert_ffn.h).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "bsr_expert_ffn.h"
#include "bsr_experts.h"
#include "bsr_fp8_blocks.h"
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
//   8-bit forward 4096 -> 14336, E = 8       16: 101 | 127    32: 123 | 127    48: 135 | 131    64: 143 | 134    96: 204 | 143
//   8-bit forward 4096 -> 4096, E = 1        16: 9 | 40    64: 11 | 41    128: 14 | 41    256: 17 | 42    384: 31 | 43
//   8-bit forward 2064 -> 1008, E = 60       16: 32 | 42    20: 40 | 43    32: 42 | 45    48: 48 | 48    64: 53 | 51
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
constexpr TileKind kFwdFp8Tiles[] = {{1, 16, 64, 256, 512, 0.50, 0.72}, {2, 32, 64, 256, 256, 0.70, 0.57},
                                     {4, 64, 64, 256, 256, 0.87, 0.80}, {128, 128, 128, 64, 512, 0.61, 0.92}};

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
// 8-bit weights, the same, while tiles of 64 leave a quarter of the CUs without one: one row, one expert, 4096 -> 4096: 7.5 us
// against 9.2; where they do not, 64 rows of it (256 tiles) 12.4 against 11.1, one row of 60 experts, 2064 -> 1008: 32 against 30.5. And
// 32 for more than one round of tiles of 64, two a CU, of rows whose pitch C is a whole number of 4096 bytes, so that all rows of a
// tile start at the same place of such a piece (pitches beside it, 3840 and 4608, show no such difference). One row of each expert, us, 32 | 64:
//   8 experts, 4096 ->   4096 (512 tiles): 32.2 | 33.8   5120: 39.1 | 42.3   8192: 54 | 72   9728: 58 | 63   14336: 81 | 88   18432: 101 | 109
//   8 experts, 8192 ->   4096: 53 | 65   5120: 56 | 61   8192: 101 | 137   14336: 139 | 139        64 experts, 4096 -> 512: 37 | 31   1024: 51 | 57
//   8 experts, 2048 ->   4096: 18.8 | 15.0   5120: 22.8 | 20.6   8192: 33 | 30   14336: 53 | 48    64 experts, 2048 -> 1024: 35 | 29
//   8 experts, 12288 -> 5120: 81 | 88   9728: 154 | 156                                           1 expert, 4096 -> 32768: 34 | 31   65536: 59 | 60
// And 32 where a long contraction's tiles of 64 leave half of a last round empty that tiles of 32 fill: 8 experts, 14336 -> 5120 (640
// tiles) 87 | 95, 8192 (1024, no such round) 137 | 138; 6144 -> 5120 47 | 50; but 4608 -> 9728 (1216) 62 | 59, 3584 -> 5120 32.8 | 32.3.
// Where it is off: one whole round (512 tiles) of such pitches, where 64 stay, may be slower by up to a fifth or faster by as much, and one
// expert of 65536 columns, 8192 long, takes 18% more. (C that is not given: a long contraction of no such pitch.)
inline int few_cols_fp8(int mt, int64_t R, int64_t E, int64_t cols, int64_t C = (1 << 20) - 1) {
    if (mt != 1) return 64;
    const int64_t groups = std::min(E, R), tiles = groups * ((R / groups + 15) / 16) * ((cols + 63) / 64);   // of equal groups
    const int64_t rounds = (tiles + 511) / 512, halves = (2 * tiles + 511) / 512;
    return tiles <= 192 || (rounds > 1 && (C % 4096 == 0 || (C >= 5632 && halves * 21 < rounds * 40))) ? 32 : 64;
}

// Whether weights that are read once, and matrices to quantise or expand, are read (expanded ones stored) as data that is not used again
// (nt): where they (of the experts that may have rows) are as large as the memory-side cache, and rows are whole lines. What else a call
// reads stays in the caches then: 7 tokens in bf16, 4096 / 11008, the whole layer 303 us | 335 without, 16 tokens there with 3584 instead
// of 11008 136 | 145; 8-bit product of one row of 8 experts, 4096 -> 14336, 83 | 93, of 256 rows in 8 bits 104 | 110. But a smaller
// matrix may be found in that cache by the next call (256 rows of 8 experts, 4096 -> 4096, again and again 36 | 28; one token in bf16,
// k = 2, 2048 / 1024, four such layers in turn: 16.8 | 15.4), and a line that two rows or two steps share is fetched twice (20 rows of 60
// experts, 2064 -> 1008: 49 | 43).
inline bool streams(int64_t bytes, bool whole_lines) { return whole_lines && bytes >= INT64_C(1) << 28; }

// 8-bit weights: where an expert has one row tile of up to 16 mt rows, mostly.
inline bool stream_fp8(int mt, int64_t R, int64_t E, int64_t N, int64_t K) {
    const int64_t groups = std::min(E, R);
    return R <= 16 * mt * groups && streams(groups * N * K, K % 128 == 0);
}

// 8 bits on both sides: 256 x 256 tiles with 8 waves, one work-group a CU, or 128 x 128 with 4, two of them. Equal groups again; a last
// round of 256 x 256 tiles that leaves half of the CUs idle or more is taken in halves, which cost 0.65 of a round. Both sides, us (rows
// of all experts: 128 x 128 | 256 x 256):
//   4096 -> 14336, E = 8     128: 109 | 123    512: 112 | 124    1024: 141 | 128    2048: 214 | 180
//   4096 -> 4096, E = 8      512: 28 | 35    1024: 36 | 36    2048: 58 | 50    4096: 92 | 85    8192: 163 | 142
//   4096 -> 4096, E = 1      256: 23 | 30    1024: 27 | 32    2048: 38 | 37    4096: 73 | 62
//   2048 -> 1008, E = 64     1024: 24 | 31    4096: 26 | 31    8192: 43 | 33    16384: 58 | 59
inline bool wide_fp8(int64_t R, int64_t E, int64_t cols, int64_t C) {
    const TileKind small = {128, 128, 128, 128, 512, 0.72, 1.25};
    const double groups = (double)std::min(E, R), each = (double)R / groups;
    const double tiles = (E == 1 ? std::ceil(each / 256) : groups * std::max(1.0, each / 256 + 0.5)) * std::ceil((double)cols / 256);
    const double whole = std::floor(tiles / 256), rest = tiles / 256 - whole;
    const double rounds = whole + (rest == 0 ? 0.0 : rest <= 0.5 ? 0.65 : 1.0);
    return rounds * (std::ceil((double)C / 128) * 1.6 + 2.0) < tile_time(small, R, E, cols, C);
}

int32_t launch_expert_fwd_few(const ExpertShape &s, int mt, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                              uint16_t *Y, void *stream);
int32_t launch_expert_bwd_input_few(const ExpertShape &s, int mt, const uint16_t *dY, const uint16_t *W, uint16_t *dX,
                                    void *stream);
int32_t launch_expert_fwd_few_mx4(const ExpertShape &s, int mt, const uint16_t *X, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream);
int32_t launch_expert_fwd_few_fp8(const ExpertShape &s, int mt, const uint16_t *X, const uint8_t *codes,
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

int32_t launch_fp8_quantize_rows(const uint16_t *X, int64_t rows, int K, uint8_t *codes, uint8_t *scales, uint16_t *values,
                                 void *stream);
int32_t launch_fp8_quantize_blocks(const uint16_t *W, int E, int N, int K, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                   uint8_t *scales_t, void *stream);
int32_t launch_fp8_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint16_t *values, void *stream);
int32_t launch_fp8_dequantize_blocks(const uint8_t *codes, const uint8_t *scales, int E, int N, int K, uint16_t *values,
                                     void *stream);
int32_t launch_expert_fwd_fp8(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream);
int32_t launch_expert_fwd_fp8_fp8(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream);

// Kernels of the whole layer for few tokens. few: up to 8 tokens share an operand. Of the up product a wave holds `span` of the columns,
// whole lines of `values` of them, `waves` of the 16 hold all, and a unit is 8 q gate rows with their up rows for each such set; wide:
// more columns than the 16 waves hold, in several spans. rs: sets of 8 output columns of a work-group of the down product; splits: work-groups that share such columns, where there are fewer sets than CUs and
// each wave of the work-groups has a line. stream_up, stream_down: see streams().
// Both sides of the rules, us: few | not: 4 tokens on 4-bit weights, 4096 / 7168 66 | 71, 4 tokens on 32 8-bit experts, 1024 / 2048 36 | 40. q = 2
// and sets | 256 columns a wave: the same 36 | 44, 16 tokens on 32 4-bit experts, 2048 / 2048 68 | 90. rs 2 | 1: 4096 / 7168 66 | 74.
struct FfnVariant {
    bool few;
    int span, q, waves;
    bool wide;
    int rs, splits;
    bool stream_up, stream_down;
};
inline FfnVariant ffn_variant(int values, int64_t T, int64_t dim, int64_t hidden, int64_t E, int64_t k) {
    const int64_t most = std::min(E, T * k);
    const bool wide = dim > 16 * 256, many = dim <= 16 * 128 && most * ((hidden + 15) / 16) >= 256;
    const int64_t lines = (dim + values - 1) / values, each = std::max(1, 128 / values);
    int waves = many ? 4 : 16;   // as few as hold the columns and leave every CU a unit
    while (waves < 16 && (waves * each < lines || most * ((hidden + 256 / waves - 1) / (256 / waves)) < 256)) waves *= 2;
    const int64_t tiles = (dim + 7) / 8, down_lines = most * ((hidden + values - 1) / values);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>({256 / tiles, down_lines / 16, 16}));
    return {T <= 8, wide || many ? 128 : 256, many ? 2 : 1, waves, wide, dim >= 16 * 256 ? 2 : 1, (int)splits,
            streams(most * 3 * dim * hidden * 128 / values, dim % values == 0), streams(most * 3 * dim * hidden * 128 / values, hidden % values == 0)};
}
size_t expert_ffn_workspace_bytes(int T, int dim, int hidden, int E, int k);
int32_t launch_expert_ffn(const uint16_t *x, int T, int dim, int hidden, int E, int k, bool renorm, const uint16_t *router,
                          int form, const void *up, const uint8_t *up_scales, const void *down, const uint8_t *down_scales,
                          const uint16_t *up_bias, const uint16_t *down_bias, uint16_t *out, void *workspace, void *stream);

}  // namespace bsr
