// bsr_experts_gemm.hip -- bf16 products grouped by expert (include/bsr_experts.h).
//
//   out[m][n] = sum over c of A(m, c) B(n, c), for each expert e:
//     forward       m row, n output column, c input column:   A = x(row)[c], B = W[e][n][c]
//     input grad    m row, n input column, c output column:   A = dY[row][c], B = W[e][c][n]
//     weight grad   m output column, n input column, c row:   A = dY[c][m],   B = x(c)[n]
// Work-groups find their expert and rows from offsets on the device.
//
// Large products are bound by the matrix cores and, beside them, by the 64 KB a step that come through L2. 16384 tokens,
// k = 2 of 8 experts, 4096 -> 11008: 2.28 ms, 1.30 PFLOP/s, matrix cores busy 71% of the time at 1.71 GHz; one dense 16384 x
// 4096 -> 4096: 394 us, 1.40 PFLOP/s (the matrix instructions alone, on random data: 2.1). Copies that skip work, of a dense
// 16384 x 16384 -> 4096 in 1591 us: no loads in the loop 1079, no waits for loads 1579, no barrier 1518, no LDS reads 1347: the
// loads' rate, not their latency.
// Gradients of 8192 tokens, k = 2 of 8, 4096 -> 4096: input 445 us (1.23 PFLOP/s), weight 481 us (1.14), their matrix cores busy
// 65 and 56%. Ragged groups cost partly empty tiles and the last round of tiles.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_experts_tile.hpp"

namespace bsr {
namespace {

using namespace dev;

struct GemmArgs {
    const uint16_t *act, *w, *bias;
    uint16_t *out;
    const int32_t *offsets, *gather;
    int T, R, E, Nout, C;   // output columns, contraction length
};

// Forward (OB = kRows) and input gradient (OB = kCols): one BM x BN tile a work-group, or half of one (piece_of).
template <Operand OB, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN * 64, 1) void k_expert_rows(GemmArgs g, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[tile_lds<BM, BN>()];
    const RowTiles<BM> tiles(g.offsets, g.E, g.R);
    const int total = tiles.total;
    const Piece piece = piece_of<BN == 256>(blockIdx.x, total * ntiles);
    if (piece.tile < 0) return;
    const TileOrder o = tile_order(piece.tile, total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    const int col = o.col * BN + (piece.half > 0 ? BN / 2 : 0);
    if (t.n <= 0 || col >= g.Nout) return;
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0;
    const int64_t wsize = (int64_t)g.Nout * g.C;
    const Side a = g.gather ? Side{g.act, (uint32_t)((int64_t)g.T * g.C * 2), g.C, t.at, t.at + t.n, g.gather, g.R, g.T}
                            : Side{g.act + (int64_t)t.at * g.C, (uint32_t)((int64_t)t.n * g.C * 2), g.C, 0, t.n, nullptr, 0, 0};
    const Side b{g.w + e * wsize, (uint32_t)(wsize * 2), OB == kRows ? g.C : g.Nout, col, g.Nout, nullptr, 0, 0};
    const uint16_t *bias = live && g.bias ? g.bias + (int64_t)e * g.Nout + col : nullptr;
    uint16_t *out = g.out + (int64_t)t.at * g.Nout + col;
    if constexpr (BN == 256) {
        if (piece.half >= 0)
            return tile_product<kRows, OB, BM, BN / 2, 4, 2>(a, b, live ? g.C : 0, bias, out, g.Nout, t.n, g.Nout - col, smem);
    }
    tile_product<kRows, OB, BM, BN, WM, WN>(a, b, live ? g.C : 0, bias, out, g.Nout, t.n, g.Nout - col, smem);
}

// Weight gradient: one BM x BN tile of one expert's dW a work-group, over all rows of the expert. Every XCD takes an eighth
// of every expert's tiles: the experts' row counts differ, and whole experts a XCD would leave some of them idle (64
// narrow experts, 16396 rows, dW 1000 x 2048: 272 -> 155 us together with token loads a step ahead; now 130 us, at least 54 of
// them for the 262 MB of dW). The eighth is rounded up: an expert of fewer than 8 tiles leaves XCDs without one.
template <int BM, int BN, int WM, int WN, bool Gathered>
__global__ __launch_bounds__(WM *WN * 64, 1) void k_expert_weight(const uint16_t *__restrict__ dY, const uint16_t *__restrict__ X,
                                                               const int32_t *__restrict__ offsets,
                                                               const int32_t *__restrict__ gather, int T, int R, int N,
                                                               int K, uint16_t *__restrict__ dW, int mtiles, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[tile_lds<BM, BN>()];
    const int per = mtiles * ntiles, share = (per + kXCDs - 1) / kXCDs, slot = blockIdx.x / kXCDs;
    const int e = slot / share, tile = (blockIdx.x % kXCDs) * share + slot % share;
    if (tile >= per) return;
    const TileOrder o = tile_order(tile, mtiles, ntiles, kRowsTogether);
    const int lo = clamp_row(scalar_load(offsets, e), R), n = max(clamp_row(scalar_load(offsets, e + 1), R) - lo, 0);
    const Side a{dY + (int64_t)lo * N, (uint32_t)((int64_t)n * N * 2), N, o.row * BM, N, nullptr, 0, 0};
    const Side b = Gathered ? Side{X, (uint32_t)((int64_t)T * K * 2), K, o.col * BN, K, gather + lo, R - lo, T}
                            : Side{X + (int64_t)lo * K, (uint32_t)((int64_t)n * K * 2), K, o.col * BN, K, nullptr, 0, 0};
    tile_product<kCols, kCols, BM, BN, WM, WN, Gathered>(a, b, n, nullptr, dW + ((int64_t)e * N + o.row * BM) * K + o.col * BN,
                                                         K, N - o.row * BM, K - o.col * BN, smem);
}

// Bias gradient: 64 columns (whole cache lines) of one expert a work-group, 8 columns a thread and 128 threads over
// the rows; their sums meet in LDS, in a fixed order. 16396 x 1000, 64 experts: 16 us (with 32 threads over the rows: 35).
constexpr int kBiasRows = 128;

__global__ __launch_bounds__(8 * kBiasRows) void k_expert_bias(const uint16_t *__restrict__ dY,
                                                               const int32_t *__restrict__ offsets, int R, int N,
                                                               uint16_t *__restrict__ dbias) {
    __shared__ float part[kBiasRows][64 + 1];
    const int e = blockIdx.y, sub = threadIdx.x & 7, c = blockIdx.x * 64 + sub * 8, rl = threadIdx.x >> 3;
    const int lo = clamp_row(scalar_load(offsets, e), R), hi = clamp_row(scalar_load(offsets, e + 1), R);
    float s[8] = {};
    if (c < N) {
        for (int r = lo + rl; r < hi; r += kBiasRows) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(dY + (int64_t)r * N + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[2 * i] += __uint_as_float(v[i] << 16);
                s[2 * i + 1] += __uint_as_float(v[i] & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[rl][sub * 8 + i] = s[i];
    __syncthreads();
    for (int half = kBiasRows / 2; half >= 16; half >>= 1) {
        for (int i = threadIdx.x; i < half * 64; i += 8 * kBiasRows) part[i >> 6][i & 63] += part[half + (i >> 6)][i & 63];
        __syncthreads();
    }
    const int col = blockIdx.x * 64 + threadIdx.x;
    if (threadIdx.x < 64 && col < N) {
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) t += part[r][threadIdx.x];
        dbias[(int64_t)e * N + col] = to_bf16(t);
    }
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}


template <Operand OB>
int32_t launch_rows(const GemmArgs &g, int64_t bm, void *stream, const char *what) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t ntiles = (g.Nout + bm - 1) / bm, blocks = max_row_tiles(g.R, g.E, bm) * ntiles + (bm == 256 ? kPieces : 0);
    if (const int32_t bad = check_grid(blocks, 512, what)) return bad;
    if (bm == 256)
        hipLaunchKernelGGL((k_expert_rows<OB, 256, 256, 2, 4>), dim3((unsigned)blocks), dim3(512), 0, st, g, (int)ntiles);
    else
        hipLaunchKernelGGL((k_expert_rows<OB, 128, 128, 2, 2>), dim3((unsigned)blocks), dim3(256), 0, st, g, (int)ntiles);
    return launched(what);
}

}  // namespace

int32_t launch_expert_fwd(const ExpertShape &s, const uint16_t *X, const uint16_t *W, const uint16_t *bias, uint16_t *Y,
                          void *stream) {
    const int tile = best_tile(kFwdTiles, s.R, s.E, s.N, s.K);
    if (tile <= 4) return launch_expert_fwd_few(s, tile, X, W, bias, Y, stream);
    return launch_rows<kRows>({X, W, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K}, tile, stream,
                              "bsr_expert_fwd");
}

int32_t launch_expert_bwd_input(const ExpertShape &s, const uint16_t *dY, const uint16_t *W, uint16_t *dX, void *stream) {
    const int tile = best_tile(kBwdInputTiles, s.R, s.E, s.K, s.N);
    if (tile <= 4) return launch_expert_bwd_input_few(s, tile, dY, W, dX, stream);
    return launch_rows<kCols>({dY, W, nullptr, dX, s.offsets, nullptr, s.T, s.R, s.E, s.K, s.N}, tile, stream,
                              "bsr_expert_bwd_input");
}

int32_t launch_expert_bwd_weight(const ExpertShape &s, const uint16_t *dY, const uint16_t *X, uint16_t *dW,
                                 uint16_t *dbias, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    // 256 x 256 tiles from 192 of them on. dW in us, 256 x 256 | 128 x 128, with 64, 512 and 2048 rows an expert:
    //   8 experts, 4096 x 4096 (2048 tiles)   62 | 72    149 | 185   448 | 584
    //   64 experts, 1000 x 2048 (2048)        66 | 74    167 | 192   528 | 672
    //   1 expert, 4096 x 4096 (256)           10 | 11     20 | 25     58 | 76
    //   8 experts, 1280 x 1280 (200)          10 | 10     21 | 25     57 | 72
    //   1 expert, 2048 x 4096 (128)            8 | 7      16 | 12     50 | 39
    //   8 experts, 1024 x 1024 (128)           8 | 6      17 | 15     48 | 40
    //   4 experts, 1000 x 1776 (112)           9 | 8      19 | 14     50 | 40
    // Experts of few tiles, which the XCDs share unevenly, lie on the wrong side of it:
    //   64 experts, 512 x 512 (256)           19 | 11     47 | 37    148 | 123
    //   16 experts, 768 x 768 (144)           10 | 9      23 | 25     65 | 76
    const bool w = (int64_t)s.E * ((s.N + 255) / 256) * ((s.K + 255) / 256) >= 192;
    const int64_t bm = w ? 256 : 128, mt = (s.N + bm - 1) / bm, nt = (s.K + bm - 1) / bm;
    const int64_t blocks = (mt * nt + 7) / 8 * 8 * s.E;
    if (const int32_t bad = check_grid(blocks, 512, "bsr_expert_bwd_weight")) return bad;
    auto run = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(w ? 512 : 256), 0, st, dY, X, s.offsets, s.row_token, s.T,
                           s.R, s.N, s.K, dW, (int)mt, (int)nt);
    };
    if (!dW) {
        // the bias alone
    } else if (w && s.row_token) run(k_expert_weight<256, 256, 2, 4, true>);
    else if (w) run(k_expert_weight<256, 256, 2, 4, false>);
    else if (s.row_token) run(k_expert_weight<128, 128, 2, 2, true>);
    else run(k_expert_weight<128, 128, 2, 2, false>);
    if (dbias)
        hipLaunchKernelGGL(k_expert_bias, dim3((unsigned)((s.N + 63) / 64), (unsigned)s.E), dim3(8 * kBiasRows), 0, st, dY,
                           s.offsets, s.R, s.N, dbias);
    return launched("bsr_expert_bwd_weight");
}

}  // namespace bsr
