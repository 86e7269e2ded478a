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

// ------------------------------------------------------------------------------------------
// bf16 activations: one 128 x 128 tile a work-group of 4 waves, steps of 64 columns. The codes are staged as they are (64 bytes a row
// and step) and turned into bf16 fragments in registers: half-wave h of a row takes the columns 32 h .. 32 h + 31, two 16-byte reads a
// step, 8 codes a product. The scale of a step is one byte for the whole tile, whose columns are those of one block. Three stages a
// side, loads two steps ahead; two work-groups a CU. 8 experts, 4096 -> 14336, equal groups: 512 rows 153 us (3.1 TB/s of weights), 2048 rows
// 264 us (910 TFLOP/s; ragged groups 303), 16384 rows 1872 us (1030 TFLOP/s), where the same product on bf16 weights with its 256 x 256 tiles takes 230 and
// 1405: each code is expanded by the two waves that share its column, and both sides are read twice as often.
// ------------------------------------------------------------------------------------------
constexpr int kA = 128 * 128, kB = 128 * 64, kStage = kA + kB;

__global__ __launch_bounds__(256, 2) void k_fp8_rows(GemmArgs g, int ntiles) {
    constexpr int BM = 128, BN = 128, out = BM * BN * 2;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[3 * kStage > out ? 3 * kStage : out];
    const RowTiles<BM> tiles(g.offsets, g.E, g.R);
    const int total = tiles.total;
    if ((int64_t)blockIdx.x >= (int64_t)total * ntiles) return;
    const TileOrder o = tile_order(xcd_remap(blockIdx.x, total * ntiles), total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    if (t.n <= 0) return;
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, kb = (g.C + 127) / 128, nb = (g.Nout + 127) / 128, steps = live ? (g.C + 63) / 64 : 0;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave & 1) * 64, n0 = (wave >> 1) * 64, l32 = lane & 31, lh = lane >> 5;
    const uint32_t base = lds_addr(smem);

    f32x16 acc[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[r][c][v] = 0.f;

    if (steps > 0) {
        // scale bytes: lane l keeps that of the steps 2 l and 2 l + 1 of 128; waited for by itself, not with all loads of every step
        const uint8_t *ws = g.w_scales + ((int64_t)e * nb + o.col) * kb;
        int held = ws[min(lane, kb - 1)];
        Stager<kRows, BM, 4, kFrag32> ga;
        ga.init({static_cast<const uint16_t *>(g.act), (uint32_t)((int64_t)(g.gather ? g.T : g.R) * g.C * 2), g.C, t.at, t.at + t.n,
                 g.gather, g.R, g.T}, g.C);
        const int64_t wbytes = (int64_t)g.Nout * g.C;
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(static_cast<const uint8_t *>(g.w) + e * wbytes, (uint32_t)wbytes);
        // lane 4 r + p of load j takes place p of row 64 j + 16 w + r; chunk q lies at q ^ (row / 4 % 4)
        uint32_t boff[2];
        int blim[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int lr = 64 * j + 16 * wave + (lane >> 2), q = (lane & 3) ^ (lr >> 2 & 3), row = o.col * BN + lr;
            boff[j] = (uint32_t)row * (uint32_t)g.C + 16u * q;
            blim[j] = row < g.Nout ? (g.C - 16 * q + 63) / 64 : 0;
        }
        asm volatile("" : "+v"(held));
        auto issue = [&](int s) __attribute__((always_inline)) {
            const uint32_t to = base + (uint32_t)(s % 3) * kStage;
#pragma unroll
            for (int j = 0; j < 4; ++j) ga.issue(to, s, j);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                dma16(rw, to + kA + (uint32_t)(4 * j + wave) * 1024u, s < blim[j] ? boff[j] + (uint32_t)s * 64u : kPast, 0);
        };
        issue(0);
        issue(1);
        for (int s = 0; s < steps; ++s) {
            wait_vm<6, 6>(6);   // step s has landed
            __syncthreads();
            issue(s + 2);       // into the stage of step s - 1, which every wave has read
            const unsigned char *ta = smem + (s % 3) * kStage, *tb = ta + kA;
            const float scale = mx4_scale_bits(__builtin_amdgcn_readlane(held, s >> 1 & 63));
            u32x4 codes[2][2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n0 + 32 * c + l32;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    codes[c][i] = *reinterpret_cast<const u32x4 *>(tb + r * 64 + (((2 * lh + i) ^ (r >> 2 & 3)) << 4));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bf16x8 fa[2], fb[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = m0 + 32 * c + l32;
                    fa[c] = *reinterpret_cast<const bf16x8 *>(ta + r * 128 + (((4 * lh + i) ^ swz8(r)) << 4));
                    fb[c] = fp8_expand8(make_uint2(codes[c][i >> 1][2 * (i & 1)], codes[c][i >> 1][2 * (i & 1) + 1]), scale);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int r = 0; r < 2; ++r) acc[r][c] = mfma32(fb[c], fa[r], acc[r][c]);
            }
            if ((s & 127) == 127) {
                held = ws[min((s + 1) / 2 + lane, kb - 1)];
                asm volatile("" : "+v"(held));
            }
        }
        wait_vm<0, 0>(0);
    }
    store_tile<BM, BN, 2, 2>(acc, live && g.bias ? g.bias + (int64_t)e * g.Nout + o.col * BN : nullptr,
                             g.out + (int64_t)t.at * g.Nout + o.col * BN, g.Nout, t.n, g.Nout - o.col * BN, smem);
}

// ------------------------------------------------------------------------------------------
// Both sides in 8 bits, on the scaled matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4: 16 x 16 x 128 products of codes, one scale
// byte per 32 of them on each side, the same one for the four 32s of a group).
//
// What the instruction does to its sums, found with single products at all positions: the products of 8 neighbouring bytes are
// aligned to the largest of their exponents and cut at 2^-13 of it (a sum of 8 such products has 13 to 16 bits); the sums of eight
// and the accumulator are added in fp32. On normal data the result is off by 2^-20 of the sum of magnitudes (K = 4096), 2^-5 of
// what rounding to bf16 does to it. The older instructions that lose nothing (16 x 16 x 32 on fp8) run at the rate of bf16.
//
// A step is one group of 128 columns: a row's 128 bytes of codes are staged like 64 bf16 columns, lane quarter h of a fragment takes
// the chunks 2 h and 2 h + 1 on both sides. Of B two stages are held, of A a ring of units of 64 rows, a little less than three
// stages' (the scale bytes have the rest of the LDS). A wave's rows are multiplied two row tiles at a time, the next two being read
// meanwhile. Before the last two every fragment of step s is in registers, and a barrier frees its stage: beside the last two the
// loads of s + 2 go out, and the first two row tiles and, column by column as they fall free, the weights of s + 1 are read. The
// ring's spare units of A are loaded before the barrier.
// Scale bytes: rows' through LDS, a word for 4 steps (loaded in each, without a branch in the loop); weights' one uniform byte a
// step, 64 steps a load (one a lane).
// 16384 x 4096 -> 4096: 223 us, 2.47 PFLOP/s; 32768 rows of 8 experts, 4096 -> 11008: 1351 us, 2.19. Copies of the former that skip
// work, of 227: no loads 190, no LDS reads either 169, all steps' loads from the same lines 215. Fragments of a whole half step ahead,
// which leave the compiler no registers: 239. Four waves of 128 x 128 each, which read a third less from LDS but wait for it alone: 260.
// Weights straight from memory into registers, in 128 x 128 tiles (16 rows a load): twice the time of such tiles.
// ------------------------------------------------------------------------------------------
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// Chunk q of row r of a stage lies at q ^ swz_pairs(r): the 16 rows of a fragment, two chunks each, take different banks.
__device__ __forceinline__ int swz_pairs(int r) { return Stager<kRows, 64, 1, kFrag16Pairs>::swz_rows(r); }

// LDS of a tile: of A a ring of units of 64 rows, of B two stages, of A's scale bytes two pieces of 4 steps (a word a row).
template <int BM, int BN>
struct Fp8Layout {
    static constexpr int kUnits = BM / 64, kRing = BM == 256 ? 11 : 5, kUnit = 64 * 128;
    static constexpr int kB = kRing * kUnit, kS = kB + 2 * BN * 128, kStages = kS + 2 * BM * 4, kOut = BM * BN * 2;
    static constexpr int kLds = kStages > kOut ? kStages : kOut;
};

// The tile of t's rows and the columns from col. Stream: the weights' loads, see streams().
template <int BM, int BN, int WM, int WN, bool Stream>
__device__ __forceinline__ void fp8_tile(const GemmArgs &g, const Rows &t, int col, unsigned char *smem) {
    constexpr int NW = WM * WN, RT = BM / WM / 16, CT = BN / WN / 16;
    static_assert(CT == 4 && RT % 2 == 0 && BM % 64 == 0, "the schedule below");
    using L = Fp8Layout<BM, BN>;
    constexpr int U = L::kUnits, RU = L::kRing, EARLY = RU - 2 * U;   // units of a step that are loaded in the first half
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, kb = (g.C + 127) / 128, nb = (g.Nout + 127) / 128, steps = live ? kb : 0;
    const int64_t wbytes = (int64_t)g.Nout * g.C, abytes = (int64_t)(g.gather ? g.T : g.R) * g.C;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave % WM) * (BM / WM), n0 = (wave / WM) * (BN / WN);
    const uint32_t base = lds_addr(smem);

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (steps > 0) {
        // Codes: load j of a wave takes the rows 8 (wave + NW j) + lane / 8 of a side, chunk lane % 8 of 16 bytes (swizzled within
        // the row). Rows past the tile's are read (or read zeros past the matrix) and only reach outputs that do not exist.
        constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;
        const int lr = 8 * wave + (lane >> 3), chunk = (lane & 7) ^ swz_pairs(lane >> 3), left = (g.C - 16 * chunk + 127) / 128;
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(g.act, (uint32_t)abytes);
        const __amdgpu_buffer_rsrc_t rb = make_rsrc(static_cast<const uint8_t *>(g.w) + e * wbytes, (uint32_t)wbytes);
        // Weights' scale bytes: lane l keeps that of step l of 64. Waited for where they are loaded: the compiler, which cannot know
        // in the loop whether it is a step after such a load, would there wait for all loads of s + 2 in every step.
        const uint8_t *ws = g.w_scales + ((int64_t)e * nb + min((col + n0) / 128, nb - 1)) * kb;
        int held = ws[min(lane, kb - 1)];
        uint32_t aoff[LA];
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const int r = lr + 8 * NW * j;
            int src = t.at + r;
            if (g.gather) src = r < t.n ? g.gather[t.at + r] : -1;
            aoff[j] = (unsigned)src < (unsigned)(g.gather ? g.T : g.R) ? (uint32_t)src * (uint32_t)g.C + 16u * chunk : kPast;
        }
        const uint32_t boff = (uint32_t)(col + lr) * (uint32_t)g.C + 16u * chunk, bstep = 8u * NW * (uint32_t)g.C;
        auto slot = [&](int q, int u) __attribute__((always_inline)) { return (uint32_t)(q + u - (q + u >= RU ? RU : 0)) * L::kUnit; };
        auto issue_a = [&](int s, int q, int u) __attribute__((always_inline)) {   // unit u of step s, whose first unit lies at q
#pragma unroll
            for (int i = 0; i < 8 / NW; ++i) {
                const int j = u * (8 / NW) + i;
                dma16(ra, base + slot(q, u) + (uint32_t)(wave + NW * i) * 1024u, s < left ? aoff[j] + (uint32_t)s * 128u : kPast, 0);
            }
        };
        auto issue_b = [&](int s, int j) __attribute__((always_inline)) {
            const uint32_t to = base + L::kB + (uint32_t)(s & 1) * (BN * 128) + (uint32_t)(wave + NW * j) * 1024u;
            const uint32_t from = s < left ? boff + (uint32_t)j * bstep + (uint32_t)s * 128u : kPast;
            if constexpr (Stream) dma16_stream(rb, to, from);
            else dma16(rb, to, from, 0);
        };
        // rows' scale bytes of 4 steps: a word a lane, 64 rows a load (waves past BM / 64 load the same words again)
        const int arows = g.gather ? g.T : g.R, sw = wave % U, ar = sw * 64 + lane;
        const int arow = ar >= t.n ? -1 : g.gather ? g.gather[t.at + ar] : t.at + ar;
        const __amdgpu_buffer_rsrc_t rsa = make_rsrc(g.act_scales, (uint32_t)((int64_t)((g.C + 511) / 512) * arows * 4));
        const int slim = (unsigned)arow < (unsigned)arows ? steps : 0;
        auto issue_scales = [&](int s) __attribute__((always_inline)) {   // those of s and its three neighbours
            dma4(rsa, base + L::kS + (uint32_t)(s >> 2 & 1) * (BM * 4) + (uint32_t)sw * 256u,
                 (s & ~3) < slim ? ((uint32_t)(s >> 2) * (uint32_t)arows + (uint32_t)arow) * 4u : kPast);
        };

        // a lane's two chunks of a fragment, for the first row of a unit, and for column tile 0 and stage 0
        const int h = lane >> 4, l16 = lane & 15;
        const uint32_t f0 = (uint32_t)(l16 * 128 + (((2 * h) ^ swz_pairs(l16)) << 4)), f1 = f0 ^ 16u;
        const uint32_t b0 = base + L::kB + (uint32_t)n0 * 128u + f0, b1 = base + L::kB + (uint32_t)n0 * 128u + f1;
        const uint32_t lane_s = base + L::kS + (uint32_t)(m0 + l16) * 4u;
        i32x8 fa[RT], fb[CT];
        int wa[RT];
        typedef __attribute__((address_space(3))) const i32x4 lds_i32x4;
        typedef __attribute__((address_space(3))) const uint8_t lds_u8;
        auto frag = [&](uint32_t p0, uint32_t p1) __attribute__((always_inline)) {
            const i32x4 lo = *(lds_i32x4 *)p0, hi = *(lds_i32x4 *)p1;
            return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
        auto read_pair = [&](int s, int q, int pair) __attribute__((always_inline)) {   // of the step s whose first unit lies at q
            const int r0 = m0 + 32 * pair;
            const uint32_t at = base + slot(q, r0 / 64) + (uint32_t)(r0 % 64) * 128u;
            const uint32_t sb = lane_s + (uint32_t)(s >> 2 & 1) * (BM * 4) + (uint32_t)(s & 3);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fa[2 * pair + i] = frag(at + f0 + (uint32_t)(i * 2048), at + f1 + (uint32_t)(i * 2048));
                wa[2 * pair + i] = *(lds_u8 *)(sb + (uint32_t)((2 * pair + i) * 64));
            }
        };
        auto read_b = [&](int st, int c) __attribute__((always_inline)) {
            fb[c] = frag(b0 + (uint32_t)(st * (BN * 128) + c * 2048), b1 + (uint32_t)(st * (BN * 128) + c * 2048));
        };
        asm volatile("" : "+v"(held));
        issue_scales(0);
#pragma unroll
        for (int u = 0; u < U; ++u) issue_a(0, 0, u);
#pragma unroll
        for (int j = 0; j < LB; ++j) issue_b(0, j);
#pragma unroll
        for (int u = 0; u < U; ++u) issue_a(1, U, u);
#pragma unroll
        for (int j = 0; j < LB; ++j) issue_b(1, j);
        wait_vm<LA + LB, LA + LB>(0);
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CT; ++c) read_b(0, c);
        read_pair(0, 0, 0);
        for (int s = 0, q = 0;;) {   // q: unit of the ring where step s begins
            const int wb = __builtin_amdgcn_readlane(held, s & 63), st = s & 1;
            const int qn = q + U - (q + U >= RU ? RU : 0), q2 = qn + U - (qn + U >= RU ? RU : 0);
            auto product = [&](int r, int c) __attribute__((always_inline)) {
                acc[r][c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[c], fa[r], acc[r][c], 0, 0, 0, wb, 0, wa[r]);
            };
#pragma unroll
            for (int pair = 0; pair < RT / 2 - 1; ++pair) {
                read_pair(s, q, pair + 1);
                constexpr int SLOTS = RT == 8 ? 2 : 1;   // pairs beside which units go out: 1 and 2, or the only one
                if (RT < 8 || pair > 0) {
                    const int k = RT < 8 ? 0 : pair - 1;
#pragma unroll
                    for (int u = k * EARLY / SLOTS; u < (k + 1) * EARLY / SLOTS; ++u) issue_a(s + 2, q2, u);
                }
#pragma unroll
                for (int c = 0; c < CT; ++c)
#pragma unroll
                    for (int r = 2 * pair; r < 2 * pair + 2; ++r) product(r, c);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // every LDS read of step s is in registers
            wait_vm<EARLY * 8 / NW, EARLY * 8 / NW>(0);           // step s + 1 has landed
            __syncthreads();
            read_pair(s + 1, qn, 0);
            issue_scales(s + 2);
#pragma unroll
            for (int u = EARLY; u < U; ++u) issue_a(s + 2, q2, u);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
#pragma unroll
                for (int j = c * LB / CT; j < (c + 1) * LB / CT; ++j) issue_b(s + 2, j);
#pragma unroll
                for (int r = RT - 2; r < RT; ++r) product(r, c);
                read_b(st ^ 1, c);
            }
            if (++s == steps) break;
            q = qn;
            if ((s & 63) == 0) {
                held = ws[min(s + lane, kb - 1)];
                asm volatile("" : "+v"(held));
            }
        }
        wait_vm<0, 0>(0);   // the last loads (of zeros) leave the stages
    }
    store_tile<BM, BN, WM, WN>(acc, live && g.bias ? g.bias + (int64_t)e * g.Nout + col : nullptr,
                               g.out + (int64_t)t.at * g.Nout + col, g.Nout, t.n, g.Nout - col, smem);
}

template <int BM, int BN, int WM, int WN, bool Stream>
__global__ __launch_bounds__(WM *WN * 64, 1) void k_fp8_fp8(GemmArgs g, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[Fp8Layout<BM, BN>::kLds];
    const RowTiles<BM> tiles(g.offsets, g.E, g.R);
    const int total = tiles.total;
    const Piece piece = piece_of<BN == 256, true>(blockIdx.x, total * ntiles);
    if (piece.tile < 0) return;
    const TileOrder o = tile_order(piece.tile, total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    const int col = o.col * BN + (piece.half > 0 ? BN / 2 : 0);
    if (t.n <= 0 || col >= g.Nout) return;
    if constexpr (BN == 256) {
        if (piece.half >= 0) return fp8_tile<BM, BN / 2, 4, 2, Stream>(g, t, col, smem);
    }
    fp8_tile<BM, BN, WM, WN, Stream>(g, t, col, smem);
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

}  // namespace

int32_t launch_expert_fwd_fp8(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream) {
    const int tile = best_tile(kFwdFp8Tiles, s.R, s.E, s.N, s.K);
    if (tile <= 4) return launch_expert_fwd_few_fp8(s, tile, X, codes, scales, bias, Y, stream);
    const GemmArgs g{X, codes, nullptr, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const int64_t ntiles = (s.N + 127) / 128, blocks = max_row_tiles(s.R, s.E, 128) * ntiles;
    if (const int32_t bad = check_grid(blocks, 256, "bsr_expert_fwd_fp8")) return bad;
    hipLaunchKernelGGL(k_fp8_rows, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), g, (int)ntiles);
    return launched("bsr_expert_fwd_fp8");
}

int32_t launch_expert_fwd_fp8_fp8(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales, const uint8_t *codes,
                                  const uint8_t *scales, const uint16_t *bias, uint16_t *Y, void *stream) {
    const GemmArgs g{xcodes, codes, xscales, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const char *what = "bsr_expert_fwd_fp8_fp8";
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool w = wide_fp8(s.R, s.E, s.N, s.K);
    const int64_t bm = w ? 256 : 128, ntiles = (s.N + bm - 1) / bm;
    const int64_t blocks = max_row_tiles(s.R, s.E, bm) * ntiles + (w ? kPieces : 0);
    if (const int32_t bad = check_grid(blocks, 512, what)) return bad;
    if (w)
        hipLaunchKernelGGL((k_fp8_fp8<256, 256, 2, 4, false>), dim3((unsigned)blocks), dim3(512), 0, st, g, (int)ntiles);
    else
        hipLaunchKernelGGL((stream_fp8(4, s.R, s.E, s.N, s.K) ? k_fp8_fp8<128, 128, 2, 2, true> : k_fp8_fp8<128, 128, 2, 2, false>), dim3((unsigned)blocks), dim3(256), 0, st, g, (int)ntiles);
    return launched(what);
}

}  // namespace bsr
