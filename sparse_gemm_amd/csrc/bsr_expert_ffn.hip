// bsr_expert_ffn.hip -- a whole layer of experts for a few tokens (include/bsr_expert_ffn.h).
//
// Bound by the bytes of the weights of the experts that a token chose. Up to 16 tokens are one operand tile of the matrix
// cores, so every weight is read once for all of them, straight from memory into registers: a load takes 128 bytes (a whole
// line) of 8 weight rows. Lane (g = l / 16, r = l % 16) holds 16 bytes, chunk 2 g + r / 8 of row r % 8. That is an operand of
// 16 "rows" whose upper eight are the lower eight's neighbouring chunk; it is multiplied twice, by the tokens' values for the even
// and for the odd chunks, and of the two results the lower and the upper eight rows are kept. The matrix cores have time for
// twice the work, and no value is moved between lanes.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "bsr_expert_ffn.h"
#include "bsr_experts_internal.hpp"
#include "bsr_experts_tile.hpp"
#include "bsr_fp8_device.hpp"

namespace bsr {
namespace {

using namespace dev;

constexpr int kTok = BSR_EXPERT_FFN_TOKENS;
constexpr int kWaves = 8;

struct FfnArgs {
    const uint16_t *x;
    int T, dim, hidden, E, k;
    const uint16_t *router;
    const void *up, *down;
    const uint8_t *up_scales, *down_scales;
    const uint16_t *up_bias, *down_bias;
    uint16_t *out;
    float *logits;
    int32_t *index;
    float *weight;
    uint16_t *h;   // [T * k][hidden]
};

// ------------------------------------------------------------------------------------------
// logits[t][e] = x[t] . router[e], one expert a work-group
// ------------------------------------------------------------------------------------------
__global__ __launch_bounds__(256) void k_ffn_logits(FfnArgs g) {
    __shared__ float part[4][kTok];
    const int e = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float acc[kTok] = {};
    for (int c = threadIdx.x * 8; c < g.dim; c += 2048) {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(g.router + (int64_t)e * g.dim + c);
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            if (t >= g.T) break;
            const u32x4 v = *reinterpret_cast<const u32x4 *>(g.x + (int64_t)t * g.dim + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[t] = fmaf(__uint_as_float(v[j] << 16), __uint_as_float(w[j] << 16), acc[t]);
                acc[t] = fmaf(__uint_as_float(v[j] & 0xFFFF0000u), __uint_as_float(w[j] & 0xFFFF0000u), acc[t]);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) acc[t] += __shfl_xor(acc[t], d);
        if (lane == 0) part[wave][t] = acc[t];
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < g.T) g.logits[(int64_t)t * g.E + e] = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
}

// ------------------------------------------------------------------------------------------
// The experts that some token chose, in ascending order, and each token's slot in them.
// ------------------------------------------------------------------------------------------
struct Chosen {
    uint32_t bits[kMaxExperts / 32];
    uint16_t expert[kTok * kMaxSlots];
    uint8_t slot[kTok * kMaxSlots][kTok];   // [chosen expert][token]: its slot there, or kNone
    int count;
};
constexpr int kNone = 255;

__device__ __forceinline__ int place_of(const Chosen &c, int e) {   // chosen experts below e
    int n = __popc(c.bits[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < e >> 5; ++w) n += __popc(c.bits[w]);
    return n;
}

__device__ __forceinline__ void choose(const FfnArgs &g, Chosen &c) {
    const int slots = g.T * g.k;
    for (int i = threadIdx.x; i < kMaxExperts / 32; i += blockDim.x) c.bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const int e = g.index[i];
        if ((unsigned)e < (unsigned)g.E) atomicOr(&c.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        for (int w = 0; w < kMaxExperts / 32; ++w) n += __popc(c.bits[w]);
        c.count = n;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < c.count * (kTok / 4); i += blockDim.x) reinterpret_cast<uint32_t *>(c.slot)[i] = ~0u;
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += blockDim.x) {
        const int e = g.index[i];
        if ((unsigned)e >= (unsigned)g.E) continue;
        const int a = place_of(c, e);
        c.expert[a] = (uint16_t)e;   // the same value from every slot
        c.slot[a][i / g.k] = (uint8_t)(i % g.k);
    }
    __syncthreads();
}

// ------------------------------------------------------------------------------------------
// Lines of weights
// ------------------------------------------------------------------------------------------
template <int Form>
struct Line {
    static constexpr int kV = Form == BSR_WEIGHTS_BF16 ? 8 : Form == BSR_WEIGHTS_FP8 ? 16 : 32;   // values of a chunk
    static constexpr int kP = kV / 8;                                                             // products of a chunk
    static constexpr int kValues = 8 * kV;                                                        // of a line
};

// One expert's matrix [rows][cols] of a form.
template <int Form>
struct Matrix {
    __amdgpu_buffer_rsrc_t codes, scales;
    int rows, cols;
    uint32_t pitch;
    __device__ __forceinline__ Matrix(const void *p, const uint8_t *s, int e, int rows_, int cols_) : rows(rows_), cols(cols_) {
        pitch = (uint32_t)cols / Line<Form>::kV * 16u;
        const uint32_t bytes = (uint32_t)rows * pitch;
        codes = make_rsrc(static_cast<const uint8_t *>(p) + (int64_t)e * bytes, bytes);
        uint32_t sb = 0;
        if constexpr (Form == BSR_WEIGHTS_MX4) sb = (uint32_t)((cols + 255) / 256) * (uint32_t)rows * 8u;
        if constexpr (Form == BSR_WEIGHTS_FP8) sb = (uint32_t)((cols + 127) / 128) * (uint32_t)((rows + 127) / 128);
        scales = make_rsrc(s + (int64_t)e * sb, sb);
    }
};

struct Held {
    u32x4 codes;
    uint32_t byte;
};

// The line s of the rows n0 .. n0 + 7 (n0 a multiple of 8); zeros outside of the matrix.
template <int Form>
__device__ __forceinline__ Held load_line(const Matrix<Form> &m, int n0, int s) {
    const int lane = threadIdx.x & 63, r = lane & 7, chunk = 2 * (lane >> 4) + (lane >> 3 & 1);
    const uint32_t at = (uint32_t)s * 128u + (uint32_t)chunk * 16u;
    const bool in = at < m.pitch && n0 < m.rows;
    Held v;
    v.codes = __builtin_bit_cast(u32x4, buf_load16(m.codes, in ? (uint32_t)(n0 + r) * m.pitch + at : kPast, 0));
    v.byte = 0;
    if constexpr (Form == BSR_WEIGHTS_MX4)
        v.byte = __builtin_amdgcn_raw_buffer_load_b8(m.scales, in ? ((uint32_t)s * (uint32_t)m.rows + (uint32_t)(n0 + r)) * 8u + chunk : kPast, 0, 0);
    if constexpr (Form == BSR_WEIGHTS_FP8)
        v.byte = __builtin_amdgcn_raw_buffer_load_b8(m.scales, in ? (uint32_t)(n0 >> 7) * (uint32_t)((m.cols + 127) / 128) + s : kPast, 0, 0);
    return v;
}

template <int Form>
__device__ __forceinline__ bf16x8 expand(const Held &v, int p) {
    if constexpr (Form == BSR_WEIGHTS_BF16) return __builtin_bit_cast(bf16x8, v.codes);
    if constexpr (Form == BSR_WEIGHTS_FP8) return fp8_expand8(make_uint2(v.codes[2 * p], v.codes[2 * p + 1]), mx4_scale_bits(v.byte));
    return mx4_expand8(v.codes[p], mx4_scale_bits(v.byte));
}

// Values of 16 tokens' rows for product p of the even (odd = 0) or odd chunks of line s; row: byte offset of this lane's
// token (lane % 16) or kPast.
template <int Form>
__device__ __forceinline__ bf16x8 load_tokens(__amdgpu_buffer_rsrc_t x, uint32_t row, int cols, int s, int p, int odd) {
    const int lane = threadIdx.x & 63, c = s * Line<Form>::kValues + (2 * (lane >> 4) + odd) * Line<Form>::kV + 8 * p;
    return buf_load16(x, c < cols && row != kPast ? row + (uint32_t)c * 2u : kPast, 0);
}

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Partial sums of a wave: item v of lane l is weight row 4 (l / 16 % 2) + v, token l % 16; the lanes from 32 on hold the odd chunks'.
__device__ __forceinline__ f32x4 halves(f32x4 even, f32x4 odd) { return (threadIdx.x & 32) ? odd : even; }

// Sum of (row, token) over the waves' partial sums.
__device__ __forceinline__ float joined(const f32x4 (*part)[64], int row, int token) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        s += part[w][(row >> 2) * 16 + token][row & 3] + part[w][(row >> 2) * 16 + 32 + token][row & 3];
    return s;
}

// ------------------------------------------------------------------------------------------
// h: 8 gate rows and their up rows of one chosen expert a unit; the waves split the columns.
// ------------------------------------------------------------------------------------------
template <int Form>
__global__ __launch_bounds__(kWaves * 64) void k_ffn_up(FfnArgs g) {
    using L = Line<Form>;
    __shared__ Chosen chosen;
    __shared__ f32x4 part[2][kWaves][64];
    choose(g, chosen);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), token = lane & 15;
    const __amdgpu_buffer_rsrc_t x = make_rsrc(g.x, (uint32_t)(g.T * g.dim) * 2u);
    const uint32_t row = token < g.T ? (uint32_t)(token * g.dim) * 2u : kPast;
    const int tiles = g.hidden / 8, steps = (g.dim + L::kValues - 1) / L::kValues, units = chosen.count * tiles;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int a = u / tiles, n0 = u % tiles * 8, e = __builtin_amdgcn_readfirstlane(chosen.expert[a]);
        const Matrix<Form> m(g.up, g.up_scales, e, 2 * g.hidden, g.dim);
        f32x4 acc[2][2] = {};   // [gate, up][even, odd]
        for (int s = wave; s < steps; s += kWaves) {
            const Held gate = load_line<Form>(m, n0, s), up = load_line<Form>(m, g.hidden + n0, s);
#pragma unroll
            for (int p = 0; p < L::kP; ++p) {
                const bf16x8 wg = expand<Form>(gate, p), wu = expand<Form>(up, p);
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const bf16x8 v = load_tokens<Form>(x, row, g.dim, s, p, odd);
                    acc[0][odd] = mfma16(wg, v, acc[0][odd]);
                    acc[1][odd] = mfma16(wu, v, acc[1][odd]);
                }
            }
        }
        __syncthreads();   // the last unit's sums have been read
        part[0][wave][lane] = halves(acc[0][0], acc[0][1]);
        part[1][wave][lane] = halves(acc[1][0], acc[1][1]);
        __syncthreads();
        const int t = threadIdx.x >> 3, i = threadIdx.x & 7;
        if (t < g.T) {
            const int j = chosen.slot[a][t];
            if (j != kNone) {
                float gv = joined(part[0], i, t), uv = joined(part[1], i, t);
                if (g.up_bias) {
                    const uint16_t *b = g.up_bias + (int64_t)e * 2 * g.hidden + n0 + i;
                    gv += from_bf16(b[0]);
                    uv += from_bf16(b[g.hidden]);
                }
                g.h[(int64_t)(t * g.k + j) * g.hidden + n0 + i] = to_bf16(gv / (1.f + __expf(-gv)) * uv);
            }
        }
    }
}

// ------------------------------------------------------------------------------------------
// out: 16 columns a work-group, over all chosen experts; the waves split the hidden columns.
// ------------------------------------------------------------------------------------------
template <int Form>
__global__ __launch_bounds__(kWaves * 64) void k_ffn_down(FfnArgs g) {
    using L = Line<Form>;
    __shared__ Chosen chosen;
    __shared__ f32x4 part[2][kWaves][64];
    choose(g, chosen);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), token = lane & 15;
    const __amdgpu_buffer_rsrc_t h = make_rsrc(g.h, (uint32_t)(g.T * g.k) * (uint32_t)g.hidden * 2u);
    const int n0 = blockIdx.x * 16, steps = (g.hidden + L::kValues - 1) / L::kValues;
    f32x4 sum[2] = {};
    for (int a = 0; a < chosen.count; ++a) {
        const Matrix<Form> m(g.down, g.down_scales, __builtin_amdgcn_readfirstlane(chosen.expert[a]), g.dim, g.hidden);
        const int j = chosen.slot[a][token];
        const uint32_t row = j != kNone ? (uint32_t)(token * g.k + j) * (uint32_t)g.hidden * 2u : kPast;
        f32x4 acc[2][2] = {};   // [rows 0 .. 7, 8 .. 15][even, odd]
        for (int s = (wave + kWaves - a * steps % kWaves) % kWaves; s < steps; s += kWaves) {
            const Held lo = load_line<Form>(m, n0, s), hi = load_line<Form>(m, n0 + 8, s);
#pragma unroll
            for (int p = 0; p < L::kP; ++p) {
                const bf16x8 wl = expand<Form>(lo, p), wh = expand<Form>(hi, p);
#pragma unroll
                for (int odd = 0; odd < 2; ++odd) {
                    const bf16x8 v = load_tokens<Form>(h, row, g.hidden, s, p, odd);
                    acc[0][odd] = mfma16(wl, v, acc[0][odd]);
                    acc[1][odd] = mfma16(wh, v, acc[1][odd]);
                }
            }
        }
        if (j != kNone) {
            const float w = g.weight[token * g.k + j];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f32x4 v = halves(acc[i][0], acc[i][1]);
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[i][q] = fmaf(w, v[q], sum[i][q]);
            }
        }
    }
    part[0][wave][lane] = sum[0];
    part[1][wave][lane] = sum[1];
    __syncthreads();
    const int t = threadIdx.x >> 4, i = threadIdx.x & 15, n = n0 + i;
    if (t < g.T && n < g.dim) {
        float v = joined(part[i >> 3], i & 7, t);
        if (g.down_bias)
            for (int j = 0; j < g.k; ++j) {
                const int e = g.index[t * g.k + j];
                if ((unsigned)e < (unsigned)g.E) v = fmaf(g.weight[t * g.k + j], from_bf16(g.down_bias[(int64_t)e * g.dim + n]), v);
            }
        g.out[(int64_t)t * g.dim + n] = to_bf16(v);
    }
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

template <int Form>
void launch_products(const FfnArgs &g, hipStream_t st) {
    const int64_t units = (int64_t)std::min(g.E, g.T * g.k) * (g.hidden / 8);
    hipLaunchKernelGGL((k_ffn_up<Form>), dim3((unsigned)std::min<int64_t>(units, 2 * kCUs)), dim3(kWaves * 64), 0, st, g);
    hipLaunchKernelGGL((k_ffn_down<Form>), dim3((unsigned)((g.dim + 15) / 16)), dim3(kWaves * 64), 0, st, g);
}

}  // namespace

size_t expert_ffn_workspace_bytes(int T, int hidden, int E, int k) {
    return up16((size_t)T * E * 4) + 2 * up16((size_t)T * k * 4) + (size_t)T * k * hidden * 2;
}

int32_t launch_expert_ffn(const uint16_t *x, int T, int dim, int hidden, int E, int k, bool renorm, const uint16_t *router,
                          int form, const void *up, const uint8_t *up_scales, const void *down, const uint8_t *down_scales,
                          const uint16_t *up_bias, const uint16_t *down_bias, uint16_t *out, void *workspace, void *stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    FfnArgs g{x, T, dim, hidden, E, k, router, up, down, up_scales, down_scales, up_bias, down_bias, out, nullptr, nullptr, nullptr, nullptr};
    g.logits = reinterpret_cast<float *>(ws);
    ws += up16((size_t)T * E * 4);
    g.index = reinterpret_cast<int32_t *>(ws);
    ws += up16((size_t)T * k * 4);
    g.weight = reinterpret_cast<float *>(ws);
    ws += up16((size_t)T * k * 4);
    g.h = reinterpret_cast<uint16_t *>(ws);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(k_ffn_logits, dim3((unsigned)E), dim3(256), 0, st, g);
    if (const int32_t bad = launch_router_fwd(g.logits, BSR_LOGITS_F32, T, E, k, renorm, g.index, g.weight, stream)) return bad;
    if (form == BSR_WEIGHTS_BF16) launch_products<BSR_WEIGHTS_BF16>(g, st);
    else if (form == BSR_WEIGHTS_MX4) launch_products<BSR_WEIGHTS_MX4>(g, st);
    else launch_products<BSR_WEIGHTS_FP8>(g, st);
    return launched("bsr_expert_ffn");
}

}  // namespace bsr
