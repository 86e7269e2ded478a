// bsr_fp8_gemm.hip -- products grouped by expert on 8-bit weights (include/bsr_fp8_blocks.h).
//
// out[m][n] = sum over c of A(m, c) B(n, c) for each expert: m row, n output column, c input column.
#include <hip/hip_runtime.h>

#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_experts_tile.hpp"
#include "bsr_fp8_device.hpp"

namespace bsr {
namespace {

using namespace dev;

struct GemmArgs {
    const void *act, *w;
    const uint8_t *act_scales, *w_scales;
    const uint16_t *bias;
    uint16_t *out;
    const int32_t *offsets, *gather;
    int T, R, E, Nout, C;   // output columns, contraction length
};

// 8 codes of A expanded, or 8 bf16 values; zeros outside of the matrix.
template <bool Fp8Act>
__device__ __forceinline__ bf16x8 act8(const GemmArgs &g, int row, int rows, int c) {
    bf16x8 v = {};
    if (row < 0 || c >= g.C) return v;
    if constexpr (Fp8Act) {
        const uint2 q = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(g.act) + (int64_t)row * g.C + c);
        return fp8_expand8(q, mx4_scale_bits(g.act_scales[((int64_t)(c >> 9) * rows + row) * 4 + (c >> 7 & 3)]));
    } else {
        return *reinterpret_cast<const bf16x8 *>(static_cast<const uint16_t *>(g.act) + (int64_t)row * g.C + c);
    }
}

// One 16 x 16 tile a wave, operands straight from memory.
template <bool Fp8Act>
__global__ __launch_bounds__(64) void k_fp8_simple(GemmArgs g, int ntiles) {
    const RowTiles<16> tiles(g.offsets, g.E, g.R);
    if ((int64_t)blockIdx.x >= (int64_t)tiles.total * ntiles) return;
    const Rows t = tiles.find(blockIdx.x / ntiles);
    if (t.n <= 0) return;
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, lane = threadIdx.x, l16 = lane & 15, h = lane >> 4, n0 = blockIdx.x % ntiles * 16;
    const int rows = g.gather ? g.T : g.R, kb = (g.C + 127) / 128, nb = (g.Nout + 127) / 128;
    int row = l16 < t.n ? t.at + l16 : -1;
    if (row >= 0 && g.gather) {
        row = g.gather[row];
        if ((unsigned)row >= (unsigned)rows) row = -1;
    }
    const int n = n0 + l16;
    const uint8_t *w = static_cast<const uint8_t *>(g.w) + ((int64_t)e * g.Nout + n) * g.C;
    const uint8_t *ws = g.w_scales + ((int64_t)e * nb + n / 128) * kb;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (live)
        for (int c0 = 0; c0 < g.C; c0 += 32) {
            const int c = c0 + 8 * h;
            bf16x8 b = {};
            if (n < g.Nout && c < g.C) b = fp8_expand8(*reinterpret_cast<const uint2 *>(w + c), mx4_scale_bits(ws[c >> 7]));
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, act8<Fp8Act>(g, row, rows, c), acc, 0, 0, 0);
        }
    const int col = n0 + 4 * h;
    if (l16 >= t.n || col >= g.Nout) return;
    if (live && g.bias) acc = add_bias4(acc, g.bias + (int64_t)e * g.Nout + col);
    store4_bf16(g.out + (int64_t)(t.at + l16) * g.Nout + col, acc[0], acc[1], acc[2], acc[3]);
}

template <bool Fp8Act>
int32_t launch(const GemmArgs &g, void *stream, const char *what) {
    const int64_t ntiles = (g.Nout + 15) / 16, blocks = max_row_tiles(g.R, g.E, 16) * ntiles;
    if (const int32_t bad = check_grid(blocks, 64, what)) return bad;
    hipLaunchKernelGGL((k_fp8_simple<Fp8Act>), dim3((unsigned)blocks), dim3(64), 0, static_cast<hipStream_t>(stream), g, (int)ntiles);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

}  // namespace

int32_t launch_expert_fwd_fp8(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream) {
    return launch<false>({X, codes, nullptr, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K}, stream,
                         "bsr_expert_fwd_fp8");
}

int32_t launch_expert_fwd_fp8_fp8(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream) {
    return launch<true>({xcodes, codes, xscales, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K}, stream,
                        "bsr_expert_fwd_fp8_fp8");
}

}  // namespace bsr
