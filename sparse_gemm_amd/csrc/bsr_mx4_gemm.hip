// bsr_mx4_gemm.hip -- products grouped by expert on microscaled 4-bit weights (include/bsr_mx4.h).
//
// out[m][n] = sum over c of A(m, c) B(n, c) for each expert: m row, n output column, c input column.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_experts_tile.hpp"
#include "bsr_mx4_device.hpp"

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
// bf16 activations: one 128 x 128 tile a work-group of 4 waves, steps of 64 columns. The codes are staged as they
// are (32 bytes a row and step) and turned into bf16 fragments in registers: half-wave h of a row takes the
// group of columns 32 h .. 32 h + 31, one 16-byte read a step whose word i is its operand of the i-th product, so
// the activation fragments take the columns 32 h + 8 i + 0 .. 7. Three stages a side, loads two steps ahead; two
// work-groups a CU. 2048 rows, 8 experts, 4096 -> 14336: 295 us, 815 TFLOP/s, matrix cores busy 48% of the time: each code is expanded
// by the two waves that share its column, and the tile is the small one. In 16 x 16 x 32 products, which read LDS and convert more for
// a product: 288 us against 278 at that time.
// ------------------------------------------------------------------------------------------
constexpr int kA = 128 * 128, kB = 128 * 32, kS = 128 * 8, kStage = kA + kB + kS;

__global__ __launch_bounds__(256, 2) void k_mx4_rows(GemmArgs g, int ntiles) {
    constexpr int BM = 128, BN = 128, out = BM * BN * 2;
    __shared__ __attribute__((aligned(1024))) unsigned char smem[3 * kStage > out ? 3 * kStage : out];
    const RowTiles<BM> tiles(g.offsets, g.E, g.R);
    const int total = tiles.total;
    if ((int64_t)blockIdx.x >= (int64_t)total * ntiles) return;
    const TileOrder o = tile_order(xcd_remap(blockIdx.x, total * ntiles), total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    if (t.n <= 0) return;
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, kb = (g.C + 255) / 256, steps = live ? (g.C + 63) / 64 : 0;
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
        Stager<kRows, BM, 4, kFrag32> ga;
        ga.init({static_cast<const uint16_t *>(g.act), (uint32_t)((int64_t)(g.gather ? g.T : g.R) * g.C * 2), g.C, t.at, t.at + t.n,
                 g.gather, g.R, g.T}, g.C);
        const int64_t wbytes = (int64_t)g.Nout * (g.C / 2);
        const __amdgpu_buffer_rsrc_t rw = make_rsrc(static_cast<const uint8_t *>(g.w) + e * wbytes, (uint32_t)wbytes);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(g.w_scales + (int64_t)e * kb * g.Nout * 8, (uint32_t)((int64_t)kb * g.Nout * 8));
        // lane 2 r + h of wave w loads the h-th group's codes and, every fourth step, the h-th scale word of row 32 w + r
        const int row = o.col * BN + wave * 32 + (lane >> 1), h = lane & 1;
        const uint32_t boff = (uint32_t)row * (uint32_t)(g.C / 2) + 16u * h, soff = (uint32_t)row * 8u + 4u * h;
        const int blim = row < g.Nout ? (g.C / 2 - 16 * h + 31) / 32 : 0, slim = row < g.Nout ? steps : 0;
        auto issue = [&](int s) __attribute__((always_inline)) {
            const uint32_t to = base + (uint32_t)(s % 3) * kStage;
#pragma unroll
            for (int j = 0; j < 4; ++j) ga.issue(to, s, j);
            dma16(rw, to + kA + (uint32_t)wave * 1024u, s < blim ? boff + (uint32_t)s * 32u : kPast, 0);
            dma4(rs, to + kA + kB + (uint32_t)wave * 256u, s < slim ? soff + (uint32_t)(s >> 2) * (uint32_t)g.Nout * 8u : kPast);
        };
        issue(0);
        issue(1);
        for (int s = 0; s < steps; ++s) {
            wait_vm<6, 6>(6);   // step s has landed
            __syncthreads();
            issue(s + 2);       // into the stage of step s - 1, which every wave has read
            const unsigned char *ta = smem + (s % 3) * kStage, *tb = ta + kA, *ts = tb + kB;
            u32x4 codes[2];
            float scale[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = n0 + 32 * c + l32;
                codes[c] = *reinterpret_cast<const u32x4 *>(tb + r * 32 + 16 * lh);
                const uint32_t byte = *(ts + r * 8 + 2 * (s & 3) + lh);
                scale[c] = mx4_scale_bits((2 * s + lh) * 32 < g.C ? byte : 0);   // bytes past K may hold anything
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bf16x8 fa[2], fb[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = m0 + 32 * c + l32;
                    fa[c] = *reinterpret_cast<const bf16x8 *>(ta + r * 128 + (((4 * lh + i) ^ swz8(r)) << 4));
                    fb[c] = mx4_expand8(codes[c][i], scale[c]);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int r = 0; r < 2; ++r) acc[r][c] = mfma32(fb[c], fa[r], acc[r][c]);
            }
        }
        wait_vm<0, 0>(0);
    }
    store_tile<BM, BN, 2, 2>(acc, live && g.bias ? g.bias + (int64_t)e * g.Nout + o.col * BN : nullptr,
                             g.out + (int64_t)t.at * g.Nout + o.col * BN, g.Nout, t.n, g.Nout - o.col * BN, smem);
}

// ------------------------------------------------------------------------------------------
// Both sides in 4 bits, on the scaled matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4: 16 x 16 x 128 products
// of codes, one scale byte per 32 of them on each side, fp32 sums).
//
// Steps of 256 columns: a row's 128 bytes of codes are staged exactly like 64 bf16 columns (8 chunks of 16
// bytes, one group each), its 8 scale bytes beside them. Lane quarter h of a fragment takes the groups 2 h + j, j = 0, 1 being the
// step's two chunks, so that its two scale bytes are one 16-bit word whose byte j the products of chunk j select. Two stages
// a side; as in the bf16 products the fragments of one chunk are read while the other is multiplied, and a barrier between them
// ends the reads of step s: the loads of step s + 2 are issued in its second chunk.
// 16384 rows, 8 experts, 4096 -> 4096: 170 us, 3.2 PFLOP/s; 32768 rows, 4096 -> 11008: 818 us, 3.6; matrix cores busy 38 and 44% of the
// time. With 32 x 32 x 64 products, before: 171 and 840 against 161 and 790 (the instructions alone, on random data, 6.4 against 7.3
// PFLOP/s). Copies of that former kernel that skip work, of 836: no loads in the loop 700, no LDS reads 744, neither 632, a single
// step 215: starts and ends of tiles and the matrix cores themselves held most of it.
// ------------------------------------------------------------------------------------------
typedef int codes_x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ codes_x8 codes8(i32x4 v) { return codes_x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <int J>
__device__ __forceinline__ f32x4 mfma_mx4(i32x4 a, i32x4 b, f32x4 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(a), codes8(b), c, 4, 4, J, sa, J, sb);
}

template <int BM, int BN>
constexpr int mx4_lds() {
    const int stages = 2 * (BM + BN) * 136, out = BM * BN * 2;
    return stages > out ? stages : out;
}

// The tile of t's rows and the columns from col.
template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void mx4_tile(const GemmArgs &g, const Rows &t, int col, unsigned char *smem) {
    constexpr int NW = WM * WN, RT = BM / WM / 16, CT = BN / WN / 16;
    static_assert(BM == NW * 32 && BN <= NW * 32 && CT == 4, "one load of scales a wave and side");
    constexpr int AB = BM * 128, BB = BN * 128, AS = 2 * (AB + BB), BS = AS + 2 * BM * 8;   // LDS: A, B, scales of A, of B
    const bool live = t.e < g.E;
    const int e = live ? t.e : 0, kb = (g.C + 255) / 256, steps = live ? kb : 0;
    const int64_t wbytes = (int64_t)g.Nout * (g.C / 2), abytes = (int64_t)(g.gather ? g.T : g.R) * (g.C / 2);

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave % WM) * (BM / WM), n0 = (wave / WM) * (BN / WN), lh = lane >> 5;
    const uint32_t base = lds_addr(smem);

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (steps > 0) {
        // codes: 16-bit units, 128 bytes a row and step
        Stager<kRows, BM, NW, kFrag16Pairs> ga;
        Stager<kRows, BN, NW, kFrag16Pairs> gb;
        constexpr int LB = Stager<kRows, BN, NW, kFrag16Pairs>::kLoads;
        ga.init({static_cast<const uint16_t *>(g.act), (uint32_t)abytes, g.C / 4, t.at, t.at + t.n, g.gather, g.R, g.T}, g.C / 4);
        gb.init({static_cast<const uint16_t *>(g.w) + e * (wbytes / 2), (uint32_t)wbytes, g.C / 4, col, g.Nout, nullptr, 0,
                 0}, g.C / 4);
        // scale words: lane 2 r + h of wave w loads word h of row 32 w + r
        const int arows = g.gather ? g.T : g.R, half = lane & 1;
        const __amdgpu_buffer_rsrc_t rsa = make_rsrc(g.act_scales, (uint32_t)((int64_t)kb * arows * 8));
        const __amdgpu_buffer_rsrc_t rsb = make_rsrc(g.w_scales + (int64_t)e * kb * g.Nout * 8, (uint32_t)((int64_t)kb * g.Nout * 8));
        // (with fewer than 32 columns a wave, two waves load the same words)
        const int ar = wave * 32 + (lane >> 1), bw = wave % (BN / 32), br = col + bw * 32 + (lane >> 1);
        const int arow = ar >= t.n ? -1 : g.gather ? g.gather[t.at + ar] : t.at + ar;
        const int sa_lim = (unsigned)arow < (unsigned)arows ? steps : 0, sb_lim = br < g.Nout ? steps : 0;
        const uint32_t sa_off = (uint32_t)arow * 8u + 4u * half, sb_off = (uint32_t)br * 8u + 4u * half;
        const uint32_t sa_step = (uint32_t)arows * 8u, sb_step = (uint32_t)g.Nout * 8u;
        auto issue_scales = [&](int st, int s) __attribute__((always_inline)) {
            dma4(rsa, base + AS + (uint32_t)st * (BM * 8) + (uint32_t)wave * 256u, s < sa_lim ? sa_off + (uint32_t)s * sa_step : kPast);
            dma4(rsb, base + BS + (uint32_t)st * (BN * 8) + (uint32_t)bw * 256u, s < sb_lim ? sb_off + (uint32_t)s * sb_step : kPast);
        };
        auto issue_a = [&](int st, int s, int j) __attribute__((always_inline)) {
            ga.issue(base + (uint32_t)st * AB, s, j);
        };
        auto issue_b = [&](int st, int s, int j) __attribute__((always_inline)) {
            gb.issue(base + 2 * AB + (uint32_t)st * BB, s, j);
        };
        // bytes of the last step whose groups do not exist are dropped
        const int h = lane >> 4, l16 = lane & 15, left = g.C / 32 - (kb - 1) * 8 - 2 * h;   // groups of this quarter in the last step
        const uint32_t keep = left >= 2 ? 0xFFFFu : left == 1 ? 0xFFu : 0u;

        // a lane's fragment address for r = 0 and chunk 0: chunk 1 flips its lowest chunk bit
        const uint32_t lane_f = (uint32_t)(l16 * 128 + (((2 * h) ^ Stager<kRows, BM, NW, kFrag16Pairs>::swz_rows(l16)) << 4));
        const uint32_t lane_a = base + (uint32_t)m0 * 128u + lane_f, lane_b = base + 2 * AB + (uint32_t)n0 * 128u + lane_f;
        const uint32_t lane_s = base + (uint32_t)(l16 * 8 + 2 * h);
        i32x4 fa[2][RT], fb[2][CT];
        int wa[RT], wb[2][CT];   // scale bytes of the quarter's two groups: chunk j takes byte j
        auto frag = [&](uint32_t at, int r, int kc) __attribute__((always_inline)) {
            typedef __attribute__((address_space(3))) const i32x4 lds_i32x4;
            return *(lds_i32x4 *)((at ^ (uint32_t)(kc << 4)) + (uint32_t)r * 2048u);
        };
        auto scale = [&](uint32_t at, uint32_t mask) __attribute__((always_inline)) {
            typedef __attribute__((address_space(3))) const uint16_t lds_u16;
            return (int)((uint32_t)*(lds_u16 *)at & mask);
        };
        auto read_a = [&](int st, int kc, int r) __attribute__((always_inline)) { fa[kc][r] = frag(lane_a + (uint32_t)st * AB, r, kc); };
        auto read_b = [&](int st, int kc, int c) __attribute__((always_inline)) { fb[kc][c] = frag(lane_b + (uint32_t)st * BB, c, kc); };
        auto scale_a = [&](int st, uint32_t mask, int r) __attribute__((always_inline)) {
            wa[r] = scale(lane_s + (uint32_t)(AS + st * (BM * 8) + (m0 + 16 * r) * 8), mask);
        };
        auto scale_b = [&](int to, int st, uint32_t mask, int c) __attribute__((always_inline)) {
            wb[to][c] = scale(lane_s + (uint32_t)(BS + st * (BN * 8) + (n0 + 16 * c) * 8), mask);
        };
        auto load = [&](int st) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) issue_a(st, st, j);
#pragma unroll
            for (int j = 0; j < LB; ++j) issue_b(st, st, j);
            issue_scales(st, st);
        };
        load(0);
        load(1);
        wait_vm<6 + LB, 6 + LB>(6 + LB);
        __syncthreads();
        uint32_t mask = steps == 1 ? keep : 0xFFFFu;
#pragma unroll
        for (int c = 0; c < CT; ++c) read_b(0, 0, c), scale_b(0, 0, mask, c);
#pragma unroll
        for (int r = 0; r < RT; ++r) read_a(0, 0, r), scale_a(0, mask, r);
        read_a(0, 1, 0);
        read_a(0, 1, 1);
        for (int s = 0; s < steps; ++s) {
            const int st = s & 1;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r < 2) {
                    read_b(st, 1, 2 * r);
                    read_b(st, 1, 2 * r + 1);
                }
                if (r + 2 < RT) read_a(st, 1, r + 2);
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[r][c] = mfma_mx4<0>(fb[0][c], fa[0][r], acc[r][c], wb[0][c], wa[r]);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // every LDS read of step s is in registers
            wait_vm<0, 0>(0);                                     // step s + 1 has landed
            __syncthreads();
            mask = s + 1 == steps - 1 ? keep : 0xFFFFu;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r < 2) {
#pragma unroll
                    for (int c = 2 * r; c < 2 * r + 2; ++c) read_b(st ^ 1, 0, c), scale_b(1, st ^ 1, mask, c);
                }
                read_a(st ^ 1, 0, r);
#pragma unroll
                for (int j = r * 4 / RT; j < (r + 1) * 4 / RT; ++j) issue_a(st, s + 2, j);
#pragma unroll
                for (int j = r * LB / RT; j < (r + 1) * LB / RT; ++j) issue_b(st, s + 2, j);
                if (r == 0) issue_scales(st, s + 2);
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[r][c] = mfma_mx4<1>(fb[1][c], fa[1][r], acc[r][c], wb[0][c], wa[r]);
                scale_a(st ^ 1, mask, r);
                if (r >= RT - 2) read_a(st ^ 1, 1, r - (RT - 2));
            }
#pragma unroll
            for (int c = 0; c < CT; ++c) wb[0][c] = wb[1][c];
        }
        wait_vm<0, 0>(0);
    }
    store_tile<BM, BN, WM, WN>(acc, live && g.bias ? g.bias + (int64_t)e * g.Nout + col : nullptr,
                               g.out + (int64_t)t.at * g.Nout + col, g.Nout, t.n, g.Nout - col, smem);
}

template <int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM *WN * 64, 1) void k_mx4_mx4(GemmArgs g, int ntiles) {
    __shared__ __attribute__((aligned(1024))) unsigned char smem[mx4_lds<BM, BN>()];
    const RowTiles<BM> tiles(g.offsets, g.E, g.R);
    const int total = tiles.total;
    const Piece piece = piece_of<BN == 256>(blockIdx.x, total * ntiles);
    if (piece.tile < 0) return;
    const TileOrder o = tile_order(piece.tile, total, ntiles, kRowsTogether);
    const Rows t = tiles.find(o.row);
    const int col = o.col * BN + (piece.half > 0 ? BN / 2 : 0);
    if (t.n <= 0 || col >= g.Nout) return;
    if constexpr (BN == 256) {
        if (piece.half >= 0) return mx4_tile<BM, BN / 2, 4, 2>(g, t, col, smem);
    }
    mx4_tile<BM, BN, WM, WN>(g, t, col, smem);
}


int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

// 256 x 256 tiles with 8 waves where the groups fill them, else 128 x 128 with 4, two work-groups a CU. 16384 rows of 8
// experts, 4096 -> 4096: 161 us against 190; one row each of 8 experts, 4096 -> 14336 (250 MB of weights): 55 us with the small tile.
bool wide(int64_t R, int64_t E, int64_t cols) { return R >= 192 * E && (R / 256 + 1) * ((cols + 255) / 256) >= 192; }

}  // namespace

int32_t launch_expert_fwd_mx4(const ExpertShape &s, const uint16_t *X, const uint8_t *codes, const uint8_t *scales,
                              const uint16_t *bias, uint16_t *Y, void *stream) {
    const int tile = best_tile(kFwdMx4Tiles, s.R, s.E, s.N, s.K);
    if (tile <= 4) return launch_expert_fwd_few_mx4(s, tile, X, codes, scales, bias, Y, stream);
    const GemmArgs g{X, codes, nullptr, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const int64_t ntiles = (s.N + 127) / 128, blocks = max_row_tiles(s.R, s.E, 128) * ntiles;
    if (const int32_t bad = check_grid(blocks, 512, "bsr_expert_fwd_mx4")) return bad;
    hipLaunchKernelGGL(k_mx4_rows, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), g, (int)ntiles);
    return launched("bsr_expert_fwd_mx4");
}

int32_t launch_expert_fwd_mx4_mx4(const ExpertShape &s, const uint8_t *xcodes, const uint8_t *xscales,
                                  const uint8_t *codes, const uint8_t *scales, const uint16_t *bias, uint16_t *Y,
                                  void *stream) {
    const GemmArgs g{xcodes, codes, xscales, scales, bias, Y, s.offsets, s.row_token, s.T, s.R, s.E, s.N, s.K};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool w = wide(s.R, s.E, s.N);
    const int64_t bm = w ? 256 : 128, ntiles = (s.N + bm - 1) / bm;
    const int64_t blocks = max_row_tiles(s.R, s.E, bm) * ntiles + (w ? kPieces : 0);
    if (const int32_t bad = check_grid(blocks, 512, "bsr_expert_fwd_mx4_mx4")) return bad;
    if (w)
        hipLaunchKernelGGL((k_mx4_mx4<256, 256, 2, 4>), dim3((unsigned)blocks), dim3(512), 0, st, g, (int)ntiles);
    else
        hipLaunchKernelGGL((k_mx4_mx4<128, 128, 2, 2>), dim3((unsigned)blocks), dim3(256), 0, st, g, (int)ntiles);
    return launched("bsr_expert_fwd_mx4_mx4");
}

}  // namespace bsr
