// bsr_experts_tile.hpp -- the pipelined tile product behind the bf16 products grouped by expert.
//
//   out[m][n] = sum over c < C of A(m, c) B(n, c)
// A work-group of NW waves owns a BM x BN tile of out and walks the contraction in steps of 64. An
// operand lies in memory either with c contiguous (kRows: one row per m or n) or with m or n
// contiguous (kCols: one row per c); both are staged as they are by direct-to-LDS loads, 4 a wave and
// step, and read as matrix-core fragments, kCols ones by transposing reads.
//   kRows tile: [BM rows][8 chunks of 16 bytes], chunk q of row r at q ^ swz_rows(r)
//   kCols tile: [64 rows][BM / 8 chunks], chunk q of row r at q ^ swz_cols(r)
// Of A three stages are held, of B two (160 KB at 256 x 256). A step is two 32-deep chunks of 16 x 16 x 32 products; while the rows of
// one chunk are multiplied, the fragments of the next are read, each into registers that a finished row has left. Between a
// step's chunks every wave waits for its LDS reads of s and for its loads of s + 1, and a barrier publishes those. The A loads of
// s + 2 are issued in the first chunk of s, the B loads, into the stage that the barrier has freed, in the second; so a load has
// one step to land, and no product waits for an LDS read right behind a barrier.
// 16 x 16 x 32 products move half of the accumulators of 32 x 32 x 16 ones per operation: alone, on random data, 2100
// TFLOP/s against 1750 at the clocks that the power allows; here, 16384 x 4096 -> 4096, 393 us against 420. Where in a chunk its reads
// and loads go is left to the compiler: with every row's reads, products and loads pinned in order 399.
#pragma once

#include <algorithm>

#include "bsr_device.hpp"

namespace bsr {
namespace dev {

enum Operand { kRows, kCols };

constexpr uint32_t kPast = 0xF0000000u;   // an offset at or past the end of every operand: such a load reads zeros

// Direct-to-LDS load of 4 bytes a lane (see dma16).
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, uint32_t m0, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(m0), "v"(voff), "s"(r)
                 : "memory", "m0");
}

// p[i] for a uniform i by a scalar load: a vector load would share the counter of the direct-to-LDS loads
// and its wait would wait for those too.
__device__ __forceinline__ int scalar_load(const int32_t *p, int i) {
    return ((const __attribute__((address_space(4))) int32_t *)(uintptr_t)p)[i];
}

// One operand of a tile: `at` is its first row (kRows) or column (kCols).
struct Side {
    const uint16_t *p;
    uint32_t bytes;          // size of the matrix behind p; loads past it read zeros
    int ld;                  // elements a row
    int at, rows;            // kRows: first row of the tile, rows that exist
    const int32_t *gather;   // row of the matrix for row i of the operand (kRows: m or n, kCols: c), or NULL
    int gcount, gmax;        // entries of gather, rows of the matrix
};

// Chunk swizzle of a kCols tile: a transposing read of 32 lanes takes rows 8 g + (0 .. 3) for two g, 32 bytes of each: row % 4
// picks a quarter of the 64 banks, g % 2 a half of that.
__device__ __forceinline__ int swz_cols(int r) { return ((r & 3) << 2) ^ (((r >> 3) & 1) << 1); }

// Frag: how the fragments of kRows tiles are read, which decides how their chunks lie: 32 rows, the half-waves a chunk each; 16 rows,
// lane quarter h chunk 4 c + h; 16 rows, quarter h chunk 2 h + c. (LDS serves 16 lanes at once, not neighbours: lanes 0 .. 3,
// 12 .. 15 and 20 .. 27, for one. With swz8 under the second kind two of them share a bank: twice the LDS cycles.)
enum Frag { kFrag32, kFrag16, kFrag16Pairs };
// Gathered: the rows of a kCols operand (c) are taken through Side::gather; kRows operands look at gather itself.
template <Operand O, int BM, int NW, Frag F, bool Gathered = false>
struct Stager {
    static __device__ __forceinline__ int swz_rows(int r) { 
        return F == kFrag32 ? swz8(r) : F == kFrag16 ? r & 7 : (r & 4) | (r & 1) << 1 | (r >> 1 & 1);
    }
    static constexpr int kLoads = BM / 8 / NW;   // 1 KB loads a wave and step
    static constexpr int kRowChunks = BM / 8, kRowsPerLoad = 64 / kRowChunks;   // kCols: a row's chunks, rows of one load
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t off[kLoads];  // byte offset of this lane's 16 bytes of load j at step 0
    uint32_t step;         // bytes between steps
    int lim[kLoads];       // steps in which load j's 16 bytes exist: from step lim[j] on it reads zeros
    // gathered kCols: rows come from the plan, 64 of them a step
    const int32_t *gather;
    int gcount, gmax, C;
    uint32_t ld2;
    uint32_t held[2];      // row offsets of this wave's tokens in kHeld steps, one a lane
    uint32_t rowoff[kLoads];   // this lane's row offset of load j of the step being issued

    __device__ __forceinline__ void init(const Side &s, int C_) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        rsrc = make_rsrc(s.p, s.bytes);
        gather = s.gather;
        gcount = s.gcount;
        gmax = s.gmax;
        C = C_;
        ld2 = (uint32_t)s.ld * 2u;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int i = place(wave, j);
            if constexpr (O == kRows) {
                const int lr = 8 * i + (lane >> 3), q = (lane & 7) ^ swz_rows(lr), row = s.at + lr;
                uint32_t src = (uint32_t)row;
                bool ok = row < s.rows;
                if (s.gather) {
                    const int t = ok ? s.gather[row] : -1;
                    ok = (unsigned)t < (unsigned)s.gmax;
                    src = (uint32_t)t;
                }
                off[j] = src * ld2 + (uint32_t)q * 16u;
                lim[j] = ok ? (C_ - 8 * q + 63) / 64 : 0;
            } else {
                const int lr = kRowsPerLoad * i + lane / kRowChunks, q = (lane % kRowChunks) ^ swz_cols(lr);
                // a column past the matrix reads the next row's values, or zeros: they only reach
                // outputs that do not exist. Rows past C read zeros by themselves.
                off[j] = (Gathered ? 0u : (uint32_t)lr * ld2) + (uint32_t)(s.at + 8 * q) * 2u;
                lim[j] = (C_ + 63) / 64;
            }
        }
        step = O == kRows ? 128u : 64u * ld2;
    }
    // Which 1 KB of the tile load j of a wave fills. kCols: a wave's loads take neighbouring rows, so that a gathered
    // operand's tokens are kWaveRows neighbouring entries of the plan.
    static constexpr int kWaveRows = kLoads * kRowsPerLoad, kHeld = 2 * 64 / kWaveRows;
    static __device__ __forceinline__ int place(int wave, int j) { return O == kRows ? wave + NW * j : kLoads * wave + j; }

    // Rows of a gathered kCols operand. hold(s), s a multiple of kHeld, takes this wave's tokens of the steps s .. s + kHeld - 1
    // by vector loads, one or two a lane, and keeps their row offsets (rows past C and tokens out of range read zeros);
    // rows(s) hands each lane those of its loads. Scalar loads of a step's tokens would return out of order
    // with the LDS reads, whose waits would then all be for everything: 8192 tokens, k = 2 of 8, 4096 -> 4096: 523 us instead of 475.
    __device__ __forceinline__ void hold(int s) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        int t[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = (s + i * (kHeld / 2) + lane / kWaveRows) * 64 + kWaveRows * wave + lane % kWaveRows;
            t[i] = gather[min(c, gcount - 1)];
            t[i] = c < C ? t[i] : -1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) held[i] = (unsigned)t[i] < (unsigned)gmax ? (uint32_t)t[i] * ld2 : kPast;
    }
    __device__ __forceinline__ void rows(int s) {
        const int lane = threadIdx.x & 63;
        const uint32_t from = s & (kHeld / 2) ? held[1] : held[0];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            rowoff[j] = (uint32_t)__builtin_amdgcn_ds_bpermute(
                4 * ((s & (kHeld / 2 - 1)) * kWaveRows + kRowsPerLoad * j + lane / kRowChunks), (int)from);
    }
    // Load j of step s into the stage at LDS byte address m0. Steps past the last one read zeros: the
    // loops issue them too, so that their bodies have no branch that products could be moved across.
    __device__ __forceinline__ void issue(uint32_t m0, int s, int j) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        uint32_t o;
        if (Gathered) o = rowoff[j] + off[j];
        else o = s < lim[j] ? off[j] + (uint32_t)s * step : kPast;
        dma16(rsrc, m0 + (uint32_t)place(wave, j) * 1024u, o, 0);
    }
    // Fragments of 16 rows / columns from t0 + 16 r and a 32-deep chunk kc of a staged tile. With t0 a multiple of 64, and of 128
    // for r above 3, r and kc only flip bits of a lane's address and add to it: it is kept once, for r = kc = 0.
    static __device__ __forceinline__ uint32_t lane_at(int t0) {
        const int lane = threadIdx.x & 63, h = lane >> 4, l16 = lane & 15;
        if constexpr (O == kRows) {
            return (uint32_t)((t0 + l16) * 128 + ((h ^ swz_rows(l16)) << 4));
        } else {
            const int R = h * 8 + (l16 >> 2), col = t0 + 4 * (l16 & 3);
            return (uint32_t)(R * (BM * 2) + ((((col >> 3) ^ swz_cols(R)) << 4) | ((col & 7) << 1)));
        }
    }
    static __device__ __forceinline__ bf16x8 frag(uint32_t at, int r, int kc) {
        if constexpr (O == kRows) {
            typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;
            return *(lds_bf16x8 *)((at ^ (uint32_t)(kc << 6)) + (uint32_t)r * 2048u);
        } else {
            const uint32_t p = (at ^ (uint32_t)(r << 5)) + (uint32_t)kc * (64u * BM);
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)p);
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4 *)(p + 8u * BM));   // 4 rows on
            const i16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(bf16x8, v);
        }
    }
};

template <int BM, int BN>
constexpr int tile_lds() {
    const int stages = 3 * BM * 128 + 2 * BN * 128, out = BM * BN * 2;
    return stages > out ? stages : out;
}

// A wave's 32 rows x 64 columns from its LDS to out: rows of 128 bytes in 16-byte pieces, piece q of row r at q ^ (r / 2 % 8), so
// that 16 rows take different banks.
__device__ __forceinline__ void store_piece(uint16_t *out, int ldo, int om, int on, const unsigned char *own) {
    const int lane = threadIdx.x & 63;
    const int q = lane & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = 8 * i + (lane >> 3);
        const u32x4 v = *reinterpret_cast<const u32x4 *>(own + m * 128 + ((q ^ ((m >> 1) & 7)) << 4));
        if (m < om && 8 * q < on) __builtin_nontemporal_store(v, reinterpret_cast<u32x4 *>(out + (int64_t)m * ldo + 8 * q));
    }
}

// Stores 32 rows x 64 columns of a wave through its 4 KB of LDS: item v of lane l of acc[t] is column 32 t + 8 (v / 4) +
// 4 (l / 32) + v % 4 of row l % 32. Bias in fp32, one rounding to bf16.
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[2], const uint16_t *bias, uint16_t *out, int ldo, int om,
                                           int on, unsigned char *own) {
    const int lane = threadIdx.x & 63, r = lane & 31, lh = lane >> 5;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            f32x4 v = quad(acc[t], q);
            const int n = 32 * t + 8 * q + 4 * lh;
            if (bias && n < on) v = add_bias4(v, bias + n);
            store4_bf16(reinterpret_cast<uint16_t *>(own + r * 128 + (((4 * t + q) ^ ((r >> 1) & 7)) << 4) + 8 * lh), v[0], v[1],
                        v[2], v[3]);
        }
    store_piece(out, ldo, om, on, own);
}

// Stores a tile from the waves' accumulators: row m of out at out + m * ldo; om rows and on (a multiple of 8) columns of
// it exist. Every wave takes its own rows through its own piece of LDS, without waiting for the others.
template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[BM / WM / 32][BN / WN / 32], const uint16_t *bias,
                                           uint16_t *out, int ldo, int om, int on, unsigned char *smem) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave % WM) * (BM / WM), n0 = (wave / WM) * (BN / WN);
    __syncthreads();   // the stages are free
#pragma unroll
    for (int r = 0; r < BM / WM / 32; ++r)
        store_rows(acc[r], bias ? bias + n0 : nullptr, out + (int64_t)(m0 + 32 * r) * ldo + n0, ldo, om - m0 - 32 * r,
                   on - n0, smem + (wave * (BM / WM / 32) + r) * 4096);
}

// The same from accumulators of 16 x 16: item v of lane l of acc[m][t] is column 16 t + 4 (l / 16) + v of row 16 m + l % 16.
__device__ __forceinline__ void store_rows(const f32x4 (&lo)[4], const f32x4 (&hi)[4], const uint16_t *bias, uint16_t *out, int ldo,
                                           int om, int on, unsigned char *own) {
    const int lane = threadIdx.x & 63, l16 = lane & 15, h = lane >> 4;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            f32x4 v = m ? hi[t] : lo[t];
            const int n = 16 * t + 4 * h, r = 16 * m + l16;
            if (bias && n < on) v = add_bias4(v, bias + n);
            store4_bf16(reinterpret_cast<uint16_t *>(own + r * 128 + (((2 * t + (h >> 1)) ^ ((r >> 1) & 7)) << 4) + 8 * (h & 1)), v[0],
                        v[1], v[2], v[3]);
        }
    store_piece(out, ldo, om, on, own);
}

template <int BM, int BN, int WM, int WN>
__device__ __forceinline__ void store_tile(const f32x4 (&acc)[BM / WM / 16][BN / WN / 16], const uint16_t *bias, uint16_t *out,
                                           int ldo, int om, int on, unsigned char *smem) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave % WM) * (BM / WM), n0 = (wave / WM) * (BN / WN);
    __syncthreads();   // the stages are free
#pragma unroll
    for (int r = 0; r < BM / WM / 32; ++r)
        store_rows(acc[2 * r], acc[2 * r + 1], bias ? bias + n0 : nullptr, out + (int64_t)(m0 + 32 * r) * ldo + n0, ldo,
                   om - m0 - 32 * r, on - n0, smem + (wave * (BM / WM / 32) + r) * 4096);
}

// The tile's product and its store. WM x WN waves, each RT x 4 accumulators of 16 x 16.
template <Operand OA, Operand OB, int BM, int BN, int WM, int WN, bool Gathered = false>
__device__ __forceinline__ void tile_product(const Side &sa, const Side &sb, int C, const uint16_t *bias, uint16_t *out,
                                             int ldo, int om, int on, unsigned char *smem) {
    constexpr int NW = WM * WN, RT = BM / WM / 16, CT = BN / WN / 16;
    static_assert(CT == 4 && RT % 4 == 0, "the schedule below");
    constexpr int AB = BM * 128, BB = BN * 128;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m0 = (wave % WM) * (BM / WM), n0 = (wave / WM) * (BN / WN);
    const uint32_t base = lds_addr(smem);

    f32x4 acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

    bf16x8 fa[2][RT], fb[2][CT];   // [chunk]
    const uint32_t lane_a = base + Stager<OA, BM, NW, kFrag16>::lane_at(m0), lane_b = base + 3 * AB + Stager<OB, BN, NW, kFrag16>::lane_at(n0);
    auto read_a = [&](int xs, int kc, int r) __attribute__((always_inline)) {
        fa[kc][r] = Stager<OA, BM, NW, kFrag16>::frag(lane_a + (uint32_t)xs * AB, r, kc);
    };
    auto read_b = [&](int vs, int kc, int t) __attribute__((always_inline)) {
        fb[kc][t] = Stager<OB, BN, NW, kFrag16>::frag(lane_b + (uint32_t)vs * BB, t, kc);
    };
    auto products = [&](int kc, int r) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[kc][t], fa[kc][r], acc[r][t], 0, 0, 0);
    };

    const int steps = (C + 63) / 64;
    if (steps > 0) {
        using StagerB = Stager<OB, BN, NW, kFrag16, Gathered>;
        Stager<OA, BM, NW, kFrag16> ga;
        StagerB gb;
        constexpr int LA = Stager<OA, BM, NW, kFrag16>::kLoads, LB = StagerB::kLoads;
        ga.init(sa, C);
        gb.init(sb, C);
        auto issue_a = [&](int xs, int s, int j) __attribute__((always_inline)) {
            ga.issue(base + (uint32_t)xs * AB, s, j);
        };
        auto issue_b = [&](int vs, int s, int j) __attribute__((always_inline)) {
            gb.issue(base + 3 * AB + (uint32_t)vs * BB, s, j);
        };
        if constexpr (Gathered) gb.hold(0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if constexpr (Gathered) gb.rows(s);
#pragma unroll
            for (int j = 0; j < LA; ++j) issue_a(s, s, j);
#pragma unroll
            for (int j = 0; j < LB; ++j) issue_b(s, s, j);
        }
        wait_vm<LA + LB, LA + LB>(LA + LB);
        __syncthreads();
#pragma unroll
        for (int t = 0; t < CT; ++t) read_b(0, 0, t);
#pragma unroll
        for (int r = 0; r < RT; ++r) read_a(0, 0, r);
        read_a(0, 1, 0);
        read_a(0, 1, 1);
        int xs = 0, vs = 0;
        for (int s = 0; s < steps; ++s) {
            const int x2 = xs == 0 ? 2 : xs - 1;   // A stage of s + 2 (that of s - 1)
            const int xn = xs == 2 ? 0 : xs + 1, vn = vs ^ 1;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r < 2) {
                    read_b(vs, 1, 2 * r);
                    read_b(vs, 1, 2 * r + 1);
                }
                if (r + 2 < RT) read_a(xs, 1, r + 2);
                if (Gathered && r == 1) gb.rows(s + 2);
#pragma unroll
                for (int j = r * LA / RT; j < (r + 1) * LA / RT; ++j) issue_a(x2, s + 2, j);
                products(0, r);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // every LDS read of step s is in registers
            wait_vm<LA, LA>(LA);                                  // all but the A loads of s + 2 have landed
            if (Gathered && (s + 3) % StagerB::kHeld == 0 && s + 3 < steps) gb.hold(s + 3);
            __syncthreads();
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if (r < 2) {
                    read_b(vn, 0, 2 * r);
                    read_b(vn, 0, 2 * r + 1);
                }
                read_a(xn, 0, r);
#pragma unroll
                for (int j = r * LB / RT; j < (r + 1) * LB / RT; ++j) issue_b(vs, s + 2, j);
                products(1, r);
                if (r >= RT - 2) read_a(xn, 1, r - (RT - 2));
            }
            xs = xn;
            vs = vn;
        }
        wait_vm<0, 0>(0);   // the last loads (of zeros) leave the stages before the output tile takes their place
    }
    store_tile<BM, BN, WM, WN>(acc, bias, out, ldo, om, on, smem);
}

// ------------------------------------------------------------------------------------------
// Rows of experts
// ------------------------------------------------------------------------------------------
struct Rows {
    int e, at, n;   // expert (E: rows past the plan), first row, rows
};

__device__ __forceinline__ int clamp_row(int v, int R) { return min(max(v, 0), R); }

// Tiles of up to BM rows, counted expert by expert; the rows past the plan come last. Lane l keeps expert l of
// the first 64: up to 64 experts offsets is read once.
template <int BM>
struct RowTiles {
    const int32_t *offsets;
    int E, R;
    int live, lo, n, upto;   // rows of all experts; this lane's expert: first row, rows, tiles up to and with it
    int total;               // tiles of the experts and of the rows past the plan

    __device__ __forceinline__ RowTiles(const int32_t *offsets_, int E_, int R_) : offsets(offsets_), E(E_), R(R_) {
        live = clamp_row(scalar_load(offsets, E), R);
        load(0);
        total = __builtin_amdgcn_readlane(upto, 63);
        for (int base = 64; base < E; base += 64) {
            RowTiles more = *this;
            more.load(base);
            total += __builtin_amdgcn_readlane(more.upto, 63);
        }
        total += tiles_of(R - live);
        total = min(total, (R + min(E + 1, R) * (BM - 1)) / BM);   // what a plan can need, whatever offsets holds
    }
    static __device__ __forceinline__ int tiles_of(int rows) { return (rows + BM - 1) / BM; }
    __device__ __forceinline__ void load(int base) {
        const int lane = threadIdx.x & 63, e = base + lane;
        lo = n = 0;
        if (e < E) {
            lo = clamp_row(offsets[e], R);
            n = max(clamp_row(offsets[e + 1], R) - lo, 0);
        }
        upto = tiles_of(n);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
    }
    // The want-th tile; n <= 0 if there is none.
    __device__ __forceinline__ Rows find(int want) const {
        RowTiles c = *this;
        for (int base = 0;;) {
            const uint64_t past = __ballot(c.upto > want);
            if (past) {
                const int l = __builtin_ctzll(past), rows = __builtin_amdgcn_readlane(c.n, l);
                const int skip = (want - (__builtin_amdgcn_readlane(c.upto, l) - tiles_of(rows))) * BM;
                return {base + l, __builtin_amdgcn_readlane(c.lo, l) + skip, min(BM, rows - skip)};
            }
            want -= __builtin_amdgcn_readlane(c.upto, 63);
            base += 64;
            if (base >= E) break;
            c.load(base);
        }
        return {E, live + want * BM, min(BM, R - live - want * BM)};
    }
};

// Row tiles that share their activations and weights in an XCD's L2: `per` of them by all column tiles.
struct TileOrder {
    int row, col;
};
__device__ __forceinline__ TileOrder tile_order(int L, int rows, int cols, int per) {
    const int chunk = L / (per * cols), r = L % (per * cols);
    const int n = min(per, rows - per * chunk);
    return {per * chunk + r % n, r / n};
}

constexpr int kRowsTogether = 4;

// Which of `tiles` tiles a block takes, one work-group a CU; -1 past the end. With Halves, where the last round would leave half of
// the CUs idle or more, its tiles are taken by two work-groups each, half of the columns a work-group (half = 0 or 1, else -1).
// Whole | halves: input gradient of 16384 rows, 8 experts, 4096 -> 4096 (4.3 rounds) 521 | 499 us; 64 experts, 2048 -> 1000
// 117 | 109; forward 32768 rows, 4096 -> 11008 (22.3 rounds) 2500 | 2460; the same in 4 bits 854 | 841 (all with 32 x 32 products).
struct Piece {
    int tile, half;
};
template <bool Halves>
__device__ __forceinline__ Piece piece_of(int64_t block, int tiles) {
    const int rest = Halves && tiles % kCUs <= kCUs / 2 ? tiles % kCUs : 0, whole = tiles - rest;
    if (block < whole) return {xcd_remap((int)block, whole), -1};
    if (block >= whole + 2 * rest) return {-1, -1};
    const int h = xcd_remap((int)block - whole, 2 * rest);
    return {whole + h / 2, h & 1};
}

}  // namespace dev

constexpr int kPieces = 128;   // work-groups that halves add to a grid: a half round

}  // namespace bsr
