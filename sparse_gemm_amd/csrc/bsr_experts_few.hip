// bsr_experts_few.hip -- grouped products for few rows an expert (decode): forward and input gradient on bf16 weights
// (include/bsr_experts.h), forward on microscaled 4-bit weights (include/bsr_mx4.h).
//
// The weights' bytes are the least that they need. A work-group owns up to 16 MT rows of one expert and BN output columns, and
// streams the BN weight rows in steps of 256 columns (512 bytes of bf16 or 128 bytes of codes a row; for the input
// gradient 2 BN bytes of 256 weight rows: whole cache lines in most cases) through a ring of NS LDS stages by
// direct-to-LDS loads, NS - 1 steps ahead. Its four waves split each step's contraction, 64 each, for all BN
// columns of the output (16 x 16 x 32 products, fp32 sums) and add their sums through LDS at the end, in a fixed
// order: with the contraction split inside the work-group, BN can be small, and a narrow layer still fills the card.
// Weights not in the caches, bytes of the experts that have rows: 8 of 8, 4096 -> 14336, one row each: in bf16 146 us, 6.4 TB/s,
// in 4 bits 51 us, 4.9 TB/s; 4 tokens, k = 2 of 8, there (5.5 experts on average) 45 us, 4.4 TB/s. 64 of 64, 4096 -> 1536, in
// bf16: 128 us, 6.3 TB/s. Nothing is read twice (219 MB counted for 7 experts' 218): the 4-bit tiles have 16 steps each in about three
// rounds of work-groups, whose starts and ends weigh. One token, k = 2 of 8, 2048 -> 1024 in bf16: 6 us, eight dependent steps.
//   bf16: lane (r = l % 16, g = l / 16) takes the columns 64 w + 32 i + 8 g + 0 .. 7 of wave w's product i
//   4-bit: the columns 64 w + 16 g + 8 i + 0 .. 7, so that its 16 codes are 8 neighbouring bytes of one group
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_experts_tile.hpp"
#include "bsr_mx4_device.hpp"

namespace bsr {
namespace {

using namespace dev;

struct FewArgs {
    const uint16_t *X;
    const void *W;
    const uint8_t *scales;   // 4-bit weights
    const uint16_t *bias;
    uint16_t *Y;
    const int32_t *offsets, *gather;
    int T, R, E, N, C;   // output columns, contraction length
};

// Weights of a tile: bf16 with the contraction contiguous (forward), bf16 with the output columns contiguous
// (input gradient), 4-bit codes with the contraction contiguous.
enum Weights { kRowsW, kColsW, kMx4W };

template <Weights W, int MT, int BN, int NS>
struct FewLayout {
    static constexpr int kM = 16 * MT;
    static constexpr int kA = kM * 512, kB = W == kMx4W ? BN * 128 : BN * 512, kS = W == kMx4W ? BN * 8 : 0;
    static constexpr int kStage = kA + kB + kS, kRed = 4 * kM * (BN + 4) * 4;
    static constexpr int kLds = NS * kStage > kRed ? NS * kStage : kRed;
    static constexpr int kALoads = 2 * MT, kBLoads = kB / 4096, kLoads = kALoads + kBLoads + (W == kMx4W ? 1 : 0);   // a wave and stage
    static constexpr int kGroups = kLds <= 80 * 1024 ? 2 : 1;   // work-groups a CU
};

// kColsW tile: [256 rows][BN / 8 chunks of 16 bytes], chunk q of row r at q ^ cswz(r): the 4 rows of a transposing
// read, and the 8 rows of two of them, fall on different banks.
template <int BN>
__device__ __forceinline__ int cswz(int r) {
    return BN == 64 ? (((r >> 1) & 1) << 1) | (((r >> 3) & 1) << 2) : ((r >> 3) & 1) << 1;
}

template <Weights W, int MT, int BN, int NS>
__global__ __launch_bounds__(256, (FewLayout<W, MT, BN, NS>::kGroups)) void k_expert_few(FewArgs g, int ntiles) {
    using L = FewLayout<W, MT, BN, NS>;
    constexpr bool MX4 = W == kMx4W, COLS = W == kColsW;
    static_assert(L::kB % 4096 == 0 && (W == kRowsW || BN == 64 || BN == 32), "whole loads a wave");
    constexpr int NT = BN / 16;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[L::kLds];
    const RowTiles<L::kM> tiles(g.offsets, g.E, g.R);
    if ((int64_t)blockIdx.x >= (int64_t)tiles.total * ntiles) return;
    const TileOrder o = tile_order(xcd_remap(blockIdx.x, tiles.total * ntiles), tiles.total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    if (t.n <= 0) return;
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, n0 = o.col * BN, steps = live ? (g.C + 255) / 256 : 0;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, gq = lane >> 4;
    const uint32_t base = lds_addr(smem);

    f32x4 acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (steps > 0) {
        const int64_t wrow = MX4 ? g.C / 2 : COLS ? (int64_t)g.N * 2 : (int64_t)g.C * 2;   // bytes of a weight row
        const int64_t wbytes = wrow * (COLS ? g.C : g.N);
        const int xrows = g.gather ? g.T : g.R;
        const __amdgpu_buffer_rsrc_t rx =
            g.gather ? make_rsrc(g.X, (uint32_t)((int64_t)xrows * g.C * 2))
                     : make_rsrc(g.X + (int64_t)t.at * g.C, (uint32_t)((int64_t)t.n * g.C * 2));   // the tile's own rows
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(static_cast<const uint8_t *>(g.W) + e * wbytes, (uint32_t)wbytes);
        // Each load: byte offset at step 0 and the number of steps in which its bytes exist.
        uint32_t aoff[L::kALoads], boff[L::kBLoads];
        int alim[L::kALoads], blim[L::kBLoads];
#pragma unroll
        for (int j = 0; j < L::kALoads; ++j) {   // 2 rows of 512 bytes a load, chunk q of row r at q ^ (r % 16)
            const int r = 2 * (wave + 4 * j) + (lane >> 5), q = (lane & 31) ^ (r & 15);
            const int src = r >= t.n ? -1 : g.gather ? g.gather[t.at + r] : r;
            aoff[j] = (uint32_t)src * (uint32_t)g.C * 2u + (uint32_t)q * 16u;
            alim[j] = (unsigned)src < (unsigned)(g.gather ? xrows : t.n) ? (g.C * 2 - 16 * q + 511) / 512 : 0;
        }
#pragma unroll
        for (int j = 0; j < L::kBLoads; ++j) {
            const int i = wave + 4 * j;
            if constexpr (COLS) {   // 512 / BN contraction rows a load
                const int r = (512 / BN) * i + lane / (BN / 8), q = (lane % (BN / 8)) ^ cswz<BN>(r);
                boff[j] = (uint32_t)r * (uint32_t)wrow + (uint32_t)(n0 + 8 * q) * 2u;
                blim[j] = n0 + 8 * q < g.N ? (g.C - r + 255) / 256 : 0;
            } else {
                const int r = MX4 ? 8 * i + (lane >> 3) : 2 * i + (lane >> 5);
                const int q = MX4 ? (lane & 7) ^ swz8(r) : (lane & 31) ^ (r & 15);
                boff[j] = (uint32_t)(n0 + r) * (uint32_t)wrow + (uint32_t)q * 16u;
                blim[j] = n0 + r >= g.N ? 0 : MX4 ? (g.C / 2 - 16 * q + 127) / 128 : (g.C * 2 - 16 * q + 511) / 512;
            }
        }
        const uint32_t bstep = MX4 ? 128u : COLS ? 256u * (uint32_t)wrow : 512u;
        // 4-bit: word h of row 32 w + r (w = wave % (BN / 32): several waves load the same words)
        const int sw = wave % (BN >= 32 ? BN / 32 : 1), kb = (g.C + 255) / 256, srow = n0 + sw * 32 + (lane >> 1);
        const __amdgpu_buffer_rsrc_t rs = MX4 ? make_rsrc(g.scales + (int64_t)e * kb * g.N * 8, (uint32_t)((int64_t)kb * g.N * 8)) : rw;
        const uint32_t soff = (uint32_t)srow * 8u + 4u * (lane & 1);
        const int slim = srow < g.N ? steps : 0;
        auto issue = [&](int s) __attribute__((always_inline)) {
            const uint32_t to = base + (uint32_t)(s % NS) * L::kStage;
#pragma unroll
            for (int j = 0; j < L::kALoads; ++j)
                dma16(rx, to + (uint32_t)(wave + 4 * j) * 1024u, s < alim[j] ? aoff[j] + (uint32_t)s * 512u : kPast, 0);
#pragma unroll
            for (int j = 0; j < L::kBLoads; ++j)
                dma16(rw, to + L::kA + (uint32_t)(wave + 4 * j) * 1024u, s < blim[j] ? boff[j] + (uint32_t)s * bstep : kPast, 0);
            if constexpr (MX4)
                dma4(rs, to + L::kA + L::kB + (uint32_t)sw * 256u, s < slim ? soff + (uint32_t)s * (uint32_t)g.N * 8u : kPast);
        };
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) issue(s);
        for (int s = 0; s < steps; ++s) {
            wait_vm<(NS - 2) * L::kLoads, (NS - 2) * L::kLoads>(0);   // step s has landed
            __syncthreads();
            const unsigned char *ta = smem + (s % NS) * L::kStage, *tb = ta + L::kA;
            bf16x8 fa[MT][2], fb[NT][2];
            uint2 codes[MX4 ? NT : 1];
            uint32_t byte[MX4 ? NT : 1];
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int q = MX4 ? wave * 8 + 2 * gq + i : wave * 8 + 4 * i + gq;
                    fa[m][i] = *reinterpret_cast<const bf16x8 *>(ta + (16 * m + r16) * 512 + ((q ^ r16) << 4));
                }
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                if constexpr (MX4) {
                    const int r = c * 16 + r16, q = 2 * wave + (gq >> 1);   // the group
                    codes[c] = *reinterpret_cast<const uint2 *>(tb + r * 128 + ((q ^ swz8(r)) << 4) + 8 * (gq & 1));
                    byte[c] = *(ta + L::kA + L::kB + r * 8 + q);
                } else if constexpr (COLS) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = 64 * wave + 32 * i + 8 * gq + (r16 >> 2), col = 16 * c + 4 * (r16 & 3);
                        auto at = [&](int row) {
                            return (lds_i16x4 *)(tb + row * (2 * BN) + ((((col >> 3) ^ cswz<BN>(row)) << 4) | ((col & 7) << 1)));
                        };
                        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(r));
                        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(at(r + 4));
                        const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                        fb[c][i] = __builtin_bit_cast(bf16x8, v);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        fb[c][i] = *reinterpret_cast<const bf16x8 *>(tb + (16 * c + r16) * 512 + (((wave * 8 + 4 * i + gq) ^ r16) << 4));
                }
            }
            issue(s + NS - 1);   // while the reads arrive; into the stage of step s - 1, which every wave has read
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                if constexpr (MX4) {   // bytes past the contraction may hold anything
                    const float scale = mx4_scale_bits((s * 8 + 2 * wave + (gq >> 1)) * 32 < g.C ? byte[c] : 0);
                    fb[c][0] = mx4_expand8(codes[c].x, scale);
                    fb[c][1] = mx4_expand8(codes[c].y, scale);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[c][i], fa[m][i], acc[m][c], 0, 0, 0);
            }
        }
        wait_vm<0, 0>(0);   // the last loads (of zeros) leave the stages
    }
    __syncthreads();

    // Item v of lane l of acc[m][c] is column 16 c + 4 (l / 16) + v of row 16 m + l % 16.
    float *red = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int c = 0; c < NT; ++c)
            *reinterpret_cast<f32x4 *>(red + (wave * L::kM + 16 * m + r16) * (BN + 4) + 16 * c + 4 * gq) = acc[m][c];
    __syncthreads();
    const int n = (threadIdx.x % (BN / 4)) * 4;
    if (n0 + n >= g.N) return;
    f32x4 b4 = {0.f, 0.f, 0.f, 0.f};
    if (live && g.bias) b4 = add_bias4(b4, g.bias + (int64_t)e * g.N + n0 + n);
    for (int m = threadIdx.x / (BN / 4); m < t.n; m += 1024 / BN) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w) v += *reinterpret_cast<const f32x4 *>(red + (w * L::kM + m) * (BN + 4) + n);
        v += b4;
        store4_bf16(g.Y + (int64_t)(t.at + m) * g.N + n0 + n, v[0], v[1], v[2], v[3]);
    }
}

template <Weights W, int MT, int BN, int NS>
int32_t launch(const FewArgs &g, void *stream, const char *what) {
    const int64_t ntiles = (g.N + BN - 1) / BN, blocks = max_row_tiles(g.R, g.E, 16 * MT) * ntiles;
    if (const int32_t bad = check_grid(blocks, 256, what)) return bad;
    hipLaunchKernelGGL((k_expert_few<W, MT, BN, NS>), dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream),
                       g, (int)ntiles);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

}  // namespace

int32_t launch_expert_fwd_few(const ExpertShape &s, int mt, const uint16_t *X, const uint16_t *W, const uint16_t *bias,
                              uint16_t *Y, void *stream) {
    const FewArgs g{X, W, nullptr, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const char *what = "bsr_expert_fwd";
    return mt == 1 ? launch<kRowsW, 1, 32, 3>(g, stream, what)
                   : mt == 2 ? launch<kRowsW, 2, 32, 4>(g, stream, what) : launch<kRowsW, 4, 32, 3>(g, stream, what);
}

int32_t launch_expert_bwd_input_few(const ExpertShape &s, int mt, const uint16_t *dY, const uint16_t *W, uint16_t *dX,
                                    void *stream) {
    const FewArgs g{dY, W, nullptr, nullptr, dX, s.offsets, nullptr, s.T, s.R, s.E, s.K, s.N};
    const char *what = "bsr_expert_bwd_input";
    if (few_cols_bwd_input(mt, s.R, s.E, s.K) == 32) return launch<kColsW, 1, 32, 3>(g, stream, what);
    return mt == 1 ? launch<kColsW, 1, 64, 3>(g, stream, what)
                   : mt == 2 ? launch<kColsW, 2, 64, 3>(g, stream, what) : launch<kColsW, 4, 64, 2>(g, stream, what);
}

int32_t launch_expert_fwd_few_mx4(const ExpertShape &s, int mt, const uint16_t *X, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream) {
    const FewArgs g{X, codes, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const char *what = "bsr_expert_fwd_mx4";
    if (few_cols_mx4(mt, s.R, s.E, s.N) == 32) return launch<kMx4W, 1, 32, 4>(g, stream, what);
    return mt == 1 ? launch<kMx4W, 1, 64, 4>(g, stream, what) : launch<kMx4W, 2, 64, 3>(g, stream, what);
}

}  // namespace bsr
