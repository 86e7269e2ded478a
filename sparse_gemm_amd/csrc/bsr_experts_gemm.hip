// bsr_experts_gemm.hip -- products grouped by expert (include/bsr_experts.h, include/bsr_mx4.h).
//
//   out[m][n] = sum over c of A(m, c) B(n, c), for each expert e:
//     forward       m row, n output column, c input column:   A = x(row)[c], B = W[e][n][c]
//     input grad    m row, n input column, c output column:   A = dY[row][c], B = W[e][c][n]
//     weight grad   m output column, n input column, c row:   A = dY[c][m],   B = x(c)[n]
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "bsr_device.hpp"
#include "bsr_experts_internal.hpp"
#include "bsr_mx4_device.hpp"

namespace bsr {
namespace {

using namespace dev;

constexpr int kBM = 128, kBN = 128, kBK = 64;
constexpr int kTileBytes = 128 * kBK * 2;
constexpr uint32_t kPast = 0xF0000000u;   // an offset past every operand: such a load reads zeros

enum Operand { kRows, kCols, kMx4 };

struct Side {
    const void *p;             // first element of this expert's / tile's matrix
    uint32_t bytes;            // its size
    const uint8_t *scales;     // kMx4
    int ld;                    // elements (kMx4: rows of the scale array)
    const int32_t *gather;     // token of each row (kRows: output rows; kCols: contraction rows), or NULL
    int gmax;                  // tokens
    int rows;                  // rows (kRows, kMx4) or columns (kCols) that exist
    int at;                    // first of them in this tile
};

// Stages the 128 x 64 tile of contraction step c0 .. c0 + 63 (of C) at LDS byte address `to`.
template <Operand O>
__device__ __forceinline__ void stage(const Side &s, int c0, int C, unsigned char *to) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (O == kMx4) {
        const int r = s.at + (threadIdx.x >> 1), g = (c0 >> 5) + (threadIdx.x & 1);
        float v[32];
        int64_t row = r < s.rows && g * 32 < C ? r : -1;
        if (row >= 0 && s.gather) {
            row = s.gather[r];
            if (row >= s.gmax) row = -1;
        }
        if (row >= 0) {
            const u32x4 codes = *reinterpret_cast<const u32x4 *>(static_cast<const uint8_t *>(s.p) + row * (C / 2) + g * 16);
            mx4_expand(codes, s.scales[((int64_t)(g >> 3) * s.ld + row) * 8 + (g & 7)], v);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
        const int lr = threadIdx.x >> 1;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = (uint32_t)to_bf16(v[8 * q + 2 * i]) | ((uint32_t)to_bf16(v[8 * q + 2 * i + 1]) << 16);
            *reinterpret_cast<u32x4 *>(to + lr * 128 + (((4 * (threadIdx.x & 1) + q) ^ swz8(lr)) << 4)) = o;
        }
        return;
    }
    const __amdgpu_buffer_rsrc_t r = make_rsrc(s.p, s.bytes);
    const uint32_t m0 = lds_addr(to);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int i = wave + 4 * j;
        uint32_t off;
        if constexpr (O == kRows) {
            const int lr = 8 * i + (lane >> 3), row = s.at + lr, c = c0 + 8 * ((lane & 7) ^ swz8(lr));
            int src = row;
            bool ok = row < s.rows && c < C;
            if (s.gather) {
                src = row < s.rows ? s.gather[row] : -1;
                ok = ok && (unsigned)src < (unsigned)s.gmax;
            }
            off = ok ? (uint32_t)src * (uint32_t)s.ld * 2u + (uint32_t)c * 2u : kPast;
        } else {
            const int lc = 4 * i + (lane >> 4), c = c0 + lc, col = s.at + 8 * ((lane & 15) ^ ((lc & 3) << 2));
            int src = c;
            bool ok = c < C && col < s.rows;
            if (s.gather) {
                src = c < C ? s.gather[c] : -1;
                ok = ok && (unsigned)src < (unsigned)s.gmax;
            }
            off = ok ? (uint32_t)src * (uint32_t)s.ld * 2u + (uint32_t)col * 2u : kPast;
        }
        dma16(r, m0 + (uint32_t)i * 1024u, off, 0);
    }
}

// Fragment of rows / columns t0 .. t0 + 31 of a staged tile for contraction chunk kc (16 deep).
template <Operand O>
__device__ __forceinline__ bf16x8 frag(const unsigned char *tile, int t0, int kc) {
    const int lane = threadIdx.x & 63;
    if constexpr (O != kCols) {
        const int r = t0 + (lane & 31);
        return *reinterpret_cast<const bf16x8 *>(tile + r * 128 + (((2 * kc + (lane >> 5)) ^ swz8(r)) << 4));
    } else {
        const int gq = lane >> 4, s16 = lane & 15;
        const int R = kc * 16 + (gq >> 1) * 8 + (s16 >> 2);
        const int col = t0 + (gq & 1) * 16 + 4 * (s16 & 3);
        auto at = [&](int row) {
            return (lds_i16x4 *)(tile + row * 256 + ((((col >> 3) ^ ((row & 3) << 2)) << 4) | ((col & 7) << 1)));
        };
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(R));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(R + 4));
        const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, v);
    }
}

// One 128 x 128 tile of out (leading dimension ldo, `om` rows and `on` columns of it exist).
template <Operand OA, Operand OB>
__device__ __forceinline__ void tile_product(const Side &a, const Side &b, int C, const uint16_t *bias, uint16_t *out,
                                             int ldo, int om, int on, unsigned char *smem) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = (wave & 1) * 64, wn = (wave >> 1) * 64;
    f32x16 acc[2][2];   // [n tile][m tile]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
    const int steps = (C + kBK - 1) / kBK;
    auto load = [&](int s) __attribute__((always_inline)) {
        unsigned char *to = smem + (s & 1) * 2 * kTileBytes;
        stage<OA>(a, s * kBK, C, to);
        stage<OB>(b, s * kBK, C, to + kTileBytes);
    };
    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
        wait_vm<0, 0>(0);
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
        const unsigned char *ta = smem + (s & 1) * 2 * kTileBytes, *tb = ta + kTileBytes;
#pragma unroll
        for (int kc = 0; kc < 4; ++kc) {
            bf16x8 fa[2], fb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[i] = frag<OA>(ta, wm + 32 * i, kc);
                fb[i] = frag<OB>(tb, wn + 32 * i, kc);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(fb[i], fa[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int m = wm + 32 * j + (lane & 31);
        if (m >= om) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = wn + 32 * i + 8 * q + 4 * (lane >> 5);
                if (n >= on) continue;
                f32x4 v = quad(acc[i][j], q);
                if (bias) v = add_bias4(v, bias + n);
                store4_bf16(out + (int64_t)m * ldo + n, v[0], v[1], v[2], v[3]);
            }
    }
}

struct Rows {
    int e, at, n;   // expert (E: rows past the plan), first row, rows
};

__device__ __forceinline__ int clamp_row(int v, int R) { return min(max(v, 0), R); }

// The `want`-th tile of up to BM rows, counted expert by expert and then over the rows past the plan;
// n = 0 if there is none.
template <int BM>
__device__ __forceinline__ Rows find_rows(const int32_t *__restrict__ offsets, int E, int R, int want) {
    const int lane = threadIdx.x & 63;
    for (int base = 0; base < E; base += 64) {
        const int e = base + lane;
        int lo = 0, n = 0;
        if (e < E) {
            lo = clamp_row(offsets[e], R);
            n = max(clamp_row(offsets[e + 1], R) - lo, 0);
        }
        const int tiles = (n + BM - 1) / BM;
        int upto = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const uint64_t past = __ballot(upto > want);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int skip = (want - (__builtin_amdgcn_readlane(upto, l) - __builtin_amdgcn_readlane(tiles, l))) * BM;
            const int nl = __builtin_amdgcn_readlane(n, l);
            return {base + l, __builtin_amdgcn_readlane(lo, l) + skip, min(BM, nl - skip)};
        }
        want -= __builtin_amdgcn_readlane(upto, 63);
    }
    const int lo = clamp_row(__builtin_amdgcn_readfirstlane(offsets[E]), R) + want * BM;
    return {E, lo, min(BM, R - lo)};
}

struct GemmArgs {
    const void *act, *w;
    const uint8_t *act_scales, *w_scales;
    const uint16_t *bias;
    uint16_t *out;
    const int32_t *offsets, *gather;
    int T, R, E, Nout, C;   // output columns, contraction length
};

// Forward and input gradient: one 128-row x 128-column tile a work-group.
template <Operand OA, Operand OB>
__global__ __launch_bounds__(256) void k_expert_rows(GemmArgs g, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[4 * kTileBytes];
    const int nt = blockIdx.x % ntiles;
    const Rows t = find_rows<kBM>(g.offsets, g.E, g.R, blockIdx.x / ntiles);
    if (t.n <= 0) return;
    const bool live = t.e < g.E;
    const int C = live ? g.C : 0;
    const int e = live ? t.e : 0;
    const int64_t wsize = (int64_t)g.Nout * g.C;
    Side a{}, b{};
    if constexpr (OA == kMx4) {
        a = {g.act, 0, g.act_scales, g.gather ? g.T : g.R, g.gather, g.T, t.at + t.n, t.at};
    } else if (g.gather) {
        a = {g.act, (uint32_t)((int64_t)g.T * g.C * 2), nullptr, g.C, g.gather, g.T, t.at + t.n, t.at};
    } else {   // the tile's own rows
        a = {static_cast<const uint16_t *>(g.act) + (int64_t)t.at * g.C, (uint32_t)((int64_t)t.n * g.C * 2), nullptr, g.C,
             nullptr, 0, t.n, 0};
    }
    if constexpr (OB == kMx4) {
        const int64_t kb = (g.C + 255) / 256;
        b = {static_cast<const uint8_t *>(g.w) + e * wsize / 2, 0, g.w_scales + e * kb * g.Nout * 8, g.Nout, nullptr, 0,
             g.Nout, nt * kBN};
    } else {
        b = {static_cast<const uint16_t *>(g.w) + e * wsize, (uint32_t)(wsize * 2), nullptr, OB == kRows ? g.C : g.Nout,
             nullptr, 0, g.Nout, nt * kBN};
    }
    tile_product<OA, OB>(a, b, C, live && g.bias ? g.bias + (int64_t)e * g.Nout + nt * kBN : nullptr,
                         g.out + (int64_t)t.at * g.Nout + nt * kBN, g.Nout, t.n, g.Nout - nt * kBN, smem);
}

// Weight gradient: one 128 x 128 tile of one expert's dW a work-group, over all rows of the expert.
__global__ __launch_bounds__(256) void k_expert_weight(const uint16_t *__restrict__ dY, const uint16_t *__restrict__ X,
                                                       const int32_t *__restrict__ offsets,
                                                       const int32_t *__restrict__ gather, int T, int R, int N, int K,
                                                       uint16_t *__restrict__ dW, int mtiles, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[4 * kTileBytes];
    const int per = mtiles * ntiles, e = blockIdx.x / per, mt = (blockIdx.x % per) / ntiles, nt = blockIdx.x % ntiles;
    const int lo = clamp_row(offsets[e], R), n = max(clamp_row(offsets[e + 1], R) - lo, 0);
    const Side a{dY + (int64_t)lo * N, (uint32_t)((int64_t)n * N * 2), nullptr, N, nullptr, 0, N, mt * kBM};
    Side b{};
    if (gather) b = {X, (uint32_t)((int64_t)T * K * 2), nullptr, K, gather + lo, T, K, nt * kBN};
    else b = {X + (int64_t)lo * K, (uint32_t)((int64_t)n * K * 2), nullptr, K, nullptr, 0, K, nt * kBN};
    tile_product<kCols, kCols>(a, b, n, nullptr, dW + ((int64_t)e * N + mt * kBM) * K + nt * kBN, K, N - mt * kBM,
                               K - nt * kBN, smem);
}

// Bias gradient: 64 columns of one expert a work-group; 8 columns a thread, 32 threads over the rows.
__global__ __launch_bounds__(256) void k_expert_bias(const uint16_t *__restrict__ dY, const int32_t *__restrict__ offsets,
                                                     int R, int N, uint16_t *__restrict__ dbias) {
    __shared__ float part[32][64];
    const int e = blockIdx.y, c = blockIdx.x * 64 + (threadIdx.x & 7) * 8, rl = threadIdx.x >> 3;
    const int lo = clamp_row(offsets[e], R), hi = clamp_row(offsets[e + 1], R);
    float s[8] = {};
    if (c < N) {
        for (int r = lo + rl; r < hi; r += 32) {
            const u32x4 v = *reinterpret_cast<const u32x4 *>(dY + (int64_t)r * N + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[2 * i] += __uint_as_float(v[i] << 16);
                s[2 * i + 1] += __uint_as_float(v[i] & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) part[rl][(threadIdx.x & 7) * 8 + i] = s[i];
    __syncthreads();
    if (threadIdx.x < 64) {
        float t = 0.f;
        for (int r = 0; r < 32; ++r) t += part[r][threadIdx.x];
        const int col = blockIdx.x * 64 + threadIdx.x;
        if (col < N) dbias[(int64_t)e * N + col] = to_bf16(t);
    }
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

// Row tiles that R rows in E groups and the rows past the plan can need.
int64_t max_row_tiles(int64_t R, int64_t E, int64_t bm) { return (R + std::min(E + 1, R) * (bm - 1)) / bm; }

template <Operand OA, Operand OB>
int32_t launch_rows(const GemmArgs &g, void *stream, const char *what) {
    const int64_t ntiles = (g.Nout + kBN - 1) / kBN, blocks = max_row_tiles(g.R, g.E, kBM) * ntiles;
    if (blocks > INT32_MAX) return fail(BSR_ERR_INVALID_ARG, std::string(what) + ": too many tiles");
    hipLaunchKernelGGL((k_expert_rows<OA, OB>), dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), g,
                       (int)ntiles);
    return launched(what);
}

}  // namespace

int32_t launch_expert_fwd(const ExpertShape &s, const uint16_t *X, const uint16_t *W, const uint16_t *bias, uint16_t *Y,
                          void *stream) {
    const GemmArgs g{X, W, nullptr, nullptr, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    return launch_rows<kRows, kRows>(g, stream, "bsr_expert_fwd");
}

int32_t launch_expert_bwd_input(const ExpertShape &s, const uint16_t *dY, const uint16_t *W, uint16_t *dX, void *stream) {
    const GemmArgs g{dY, W, nullptr, nullptr, nullptr, dX, s.offsets, nullptr, s.T, s.R, s.E, s.K, s.N};
    return launch_rows<kRows, kCols>(g, stream, "bsr_expert_bwd_input");
}

int32_t launch_expert_bwd_weight(const ExpertShape &s, const uint16_t *dY, const uint16_t *X, uint16_t *dW,
                                 uint16_t *dbias, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t mt = (s.N + kBM - 1) / kBM, nt = (s.K + kBN - 1) / kBN;
    if (mt * nt * s.E > INT32_MAX) return fail(BSR_ERR_INVALID_ARG, "bsr_expert_bwd_weight: too many tiles");
    hipLaunchKernelGGL(k_expert_weight, dim3((unsigned)(mt * nt * s.E)), dim3(256), 0, st, dY, X, s.offsets, s.row_token,
                       s.T, s.R, s.N, s.K, dW, (int)mt, (int)nt);
    if (dbias)
        hipLaunchKernelGGL(k_expert_bias, dim3((unsigned)((s.N + 63) / 64), (unsigned)s.E), dim3(256), 0, st, dY, s.offsets,
                           s.R, s.N, dbias);
    return launched("bsr_expert_bwd_weight");
}

int32_t launch_expert_fwd_mx4(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream) {
    const GemmArgs g{X, codes, nullptr, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    return launch_rows<kRows, kMx4>(g, stream, "bsr_expert_fwd_mx4");
}

int32_t launch_expert_fwd_mx4_mx4(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales,
                                  const uint8_t *codes, const uint8_t *scales, const uint16_t *bias, uint16_t *Y,
                                  void *stream) {
    const GemmArgs g{xcodes, codes, xscales, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    return launch_rows<kMx4, kMx4>(g, stream, "bsr_expert_fwd_mx4_mx4");
}

}  // namespace bsr
