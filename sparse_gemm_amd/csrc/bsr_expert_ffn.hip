// bsr_expert_ffn.hip -- a whole layer of experts for a few tokens (include/bsr_expert_ffn.h).
//
// Bound by the bytes of the weights of the experts that a token chose. Up to 16 tokens are one operand tile of the matrix
// cores, so every weight is read once for all of them, straight from memory into registers: a load takes 128 bytes (a whole
// line) of 8 weight rows. Lane (g = l / 16, r = l % 16) holds 16 bytes, chunk 2 g + r / 8 of row r % 8. That is an operand of
// 16 "rows" whose upper eight are the lower eight's neighbouring chunk; it is multiplied twice, by the tokens' values for the even
// and for the odd chunks, and of the two results the lower and the upper eight rows are kept. The matrix cores have time for
// twice the work, and no value is moved between lanes.
// 7 tokens on 8 experts in bf16, 4096 / 11008: 303 us, 6.2 TB/s; 4 tokens on 4-bit ones, 4096 / 7168: 61 to 67 us, 4.2 TB/s; 16 tokens on 64 8-bit ones,
// 2048 / 1008: 88 us, 3.9 TB/s. What does not grow with the weights (layers of 64 hidden columns, and the slope from 1024 on): 4 tokens on
// 4-bit weights, 4096 columns, 12 us for the up product (router, list, rows, weights, one after the other) and 4 for the down product, in
// bf16 there 15 and 5, 16 tokens on 64 8-bit experts 14 and 6 to 8; further weights come at 6.1 and 4.4, 7.0 and 7.1, 4.8 and 4.1 TB/s. A layer of 25 MB (one
// token, 2048 / 1024 in bf16) takes 15 us.
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
constexpr int kWaves = 16;             // of a work-group of the products: one a CU
constexpr int kThreads = kWaves * 64;
constexpr int kNone = 255;

struct FfnArgs {
    const uint16_t *x;
    int T, dim, hidden, E, k;
    int renorm, route, parts;   // route: who finds the experts (Route); parts: pieces of the logits' sums
    int waves;                  // of a set of the up product (FfnVariant)
    const uint16_t *router;
    const void *up, *down;
    const uint8_t *up_scales, *down_scales;
    const uint16_t *up_bias, *down_bias;
    uint16_t *out;
    float *logits;     // [parts][T][E]
    int32_t *index;    // [T][k]
    float *weight;     // [T][k]
    uint16_t *h;       // [T * k][hidden]
    int splits;        // work-groups that share the lines of a down tile (FfnVariant)
    float *partial;    // [splits][T][dim]
    uint32_t *done;    // of each down tile: work-groups that have stored their sums
};

// Who finds the experts: the work-groups of the up product, each for itself, from x and the router or from logits that a
// launch before has summed in pieces; or the router's kernel.
enum Route { kAllInOne, kFromLogits, kRouted };
constexpr int kMostInOne = 16;   // experts of kAllInOne

// ------------------------------------------------------------------------------------------
// Lines of weights
// ------------------------------------------------------------------------------------------
template <int Form>
struct Line {
    static constexpr int kV = Form == BSR_WEIGHTS_BF16 ? 8 : Form == BSR_WEIGHTS_FP8 ? 16 : 32;   // values of a chunk
    static constexpr int kP = kV / 8;                                                             // products of a chunk
    static constexpr int kValues = 8 * kV;                                                        // of a line
};

// The matrices [rows][cols] of a form, one an expert. Loads that are not wanted (of experts, rows or chunks that do not exist) are
// issued too, at an offset past the end: behind a branch the compiler could not count the loads in flight, and would wait for all
// of them before it uses the oldest.
template <int Form>
struct Matrix {
    const uint8_t *codes, *scales;
    uint32_t pitch, bytes, scale_bytes;   // of a row's codes, of a matrix
    int rows, blocks;                     // blocks: bytes of scales a row of 128 x 128 blocks (fp8)
    __device__ __forceinline__ Matrix(const void *p, const uint8_t *s, int rows_, int cols)
        : codes(static_cast<const uint8_t *>(p)), scales(s), rows(rows_), blocks((cols + 127) / 128) {
        pitch = (uint32_t)cols / Line<Form>::kV * 16u;
        bytes = (uint32_t)rows * pitch;
        scale_bytes = Form == BSR_WEIGHTS_MX4 ? (uint32_t)((cols + 255) / 256) * (uint32_t)rows * 8u
                                              : Form == BSR_WEIGHTS_FP8 ? (uint32_t)blocks * (uint32_t)((rows + 127) / 128) : 0u;
    }
};

// One expert of them; not live: nothing is read.
template <int Form>
struct Expert {
    __amdgpu_buffer_rsrc_t codes, scales;
    __device__ __forceinline__ Expert(const Matrix<Form> &m, int e, bool live)
        : codes(make_rsrc(m.codes + (int64_t)e * m.bytes, live ? m.bytes : 0u)),
          scales(make_rsrc(m.scales + (int64_t)e * m.scale_bytes, live ? m.scale_bytes : 0u)) {}
};

// A line that no row has: its pieces lie from 2^32 - 128 on, past every row.
constexpr int kNoLine = (1 << 25) - 1;

struct Held {
    u32x4 codes;
    uint32_t byte;
};

// A lane's piece of line s of 8 rows, from the first of them on: what stays the same for all groups of 8 rows. Lane (g = l / 16,
// r = l % 16) takes chunk 2 g + r / 8 of row r % 8.
template <int Form>
struct Piece8 {
    uint32_t code, scale;   // offsets
    bool in;                // the chunk exists
    __device__ __forceinline__ Piece8(const Matrix<Form> &m, int s) {
        const int lane = threadIdx.x & 63, r = lane & 7, chunk = 2 * (lane >> 4) + (lane >> 3 & 1);
        const uint32_t at = (uint32_t)s * 128u + (uint32_t)chunk * 16u;
        in = at < m.pitch;
        code = (uint32_t)r * m.pitch + at;
        scale = Form == BSR_WEIGHTS_MX4 ? ((uint32_t)s * (uint32_t)m.rows + (uint32_t)r) * 8u + chunk : (uint32_t)s;
    }
    // Of the 8 rows from n0 (a multiple of 8). Stream: marked as not used again (nt).
    template <bool Stream = false>
    __device__ __forceinline__ Held load(const Matrix<Form> &m, const Expert<Form> &e, int n0) const {
        Held v;
        v.codes = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(e.codes, in ? code + (uint32_t)n0 * m.pitch : kPast, 0,
                                                                                  Stream ? 2 : 0));
        v.byte = 0;
        if constexpr (Form == BSR_WEIGHTS_MX4)
            v.byte = __builtin_amdgcn_raw_buffer_load_b8(e.scales, in ? scale + (uint32_t)n0 * 8u : kPast, 0, 0);
        if constexpr (Form == BSR_WEIGHTS_FP8)
            v.byte = __builtin_amdgcn_raw_buffer_load_b8(e.scales, in ? scale + (uint32_t)(n0 >> 7) * (uint32_t)m.blocks : kPast, 0, 0);
        return v;
    }
};

template <int Form>
__device__ __forceinline__ bf16x8 expand(const Held &v, int p) {
    if constexpr (Form == BSR_WEIGHTS_BF16) return __builtin_bit_cast(bf16x8, v.codes);
    if constexpr (Form == BSR_WEIGHTS_FP8) return fp8_expand8(make_uint2(v.codes[2 * p], v.codes[2 * p + 1]), mx4_scale_bits(v.byte));
    return mx4_expand8(v.codes[p], mx4_scale_bits(v.byte));
}

// The other operand: 16 tokens' values for the even chunks and, apart, for the odd ones; or, up to 8 tokens (Few), those for the
// even chunks in the lower and for the odd chunks in the upper eight of its 16 columns: one product does for both.
template <bool Few>
struct Tokens {
    static constexpr int kN = Few ? 1 : 2;          // operands a product
    static constexpr int kOdd = Few ? 40 : 32;      // from the lane with the even chunks' sums to that with the odd chunks'
    static __device__ __forceinline__ int token() { return threadIdx.x & (Few ? 7 : 15); }
    static __device__ __forceinline__ int odd(int i) { return Few ? threadIdx.x >> 3 & 1 : i; }
};

// Operand i for product p of line s; row: byte offset of this lane's token or kPast.
template <int Form, bool Few>
__device__ __forceinline__ bf16x8 load_tokens(__amdgpu_buffer_rsrc_t x, uint32_t row, int cols, int s, int p, int i) {
    const int lane = threadIdx.x & 63, c = s * Line<Form>::kValues + (2 * (lane >> 4) + Tokens<Few>::odd(i)) * Line<Form>::kV + 8 * p;
    return buf_load16(x, c < cols && row != kPast ? row + (uint32_t)c * 2u : kPast, 0);
}

// Sums of one set of 8 rows: item v of lane l is row 4 (l / 16 % 2) + v, token l % 16 (Few: l % 8); those of the even chunks in the
// lanes below 32 (Few: and l % 16 below 8), of the odd chunks in the lanes from 32 on (Few: and l % 16 from 8 on).
template <bool Few>
struct Sums {
    f32x4 v[Tokens<Few>::kN];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < Tokens<Few>::kN; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ __forceinline__ void add(bf16x8 w, const bf16x8 (&x)[Tokens<Few>::kN]) {
#pragma unroll
        for (int i = 0; i < Tokens<Few>::kN; ++i) v[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x[i], v[i], 0, 0, 0);
    }
    __device__ __forceinline__ f32x4 all() const {
        // The wait states between a matrix instruction and a read of its result. The compiler counts them, but hipcc 7.2 left them out
        // where the instruction ends a loop and an LDS write of its result follows the loop: the old sums were written.
        f32x4 even = v[0];
        if constexpr (Few) {
            asm volatile("s_nop 15" : "+v"(even));
            return even;
        }
        f32x4 odd = v[Tokens<Few>::kN - 1];   // (a choice between the places of the two would put both into memory)
        asm volatile("s_nop 15" : "+v"(even), "+v"(odd));
        const bool upper = threadIdx.x & 32;
        return f32x4{upper ? odd[0] : even[0], upper ? odd[1] : even[1], upper ? odd[2] : even[2], upper ? odd[3] : even[3]};
    }
};

// The waves' sums of one set of 8 rows. A group of 16 lanes joins 4 rows of one token: lane w takes those of wave w, 65 vectors apart
// so that the 16 take different banks, and four exchanges add them up, in an order that is the same for every lane. With one
// thread a sum, 32 reads each, the join took longer than the weights of a unit.
// Where the waves are sets of 4 or 8 that hold other rows each, the lanes of a set join its rows.
typedef f32x4 Part[kWaves][65];

template <bool Few>
struct Group {
    static constexpr int kCount = Few ? 16 : 32;   // of a set
    int token, quad;                               // rows 4 quad .. 4 quad + 3
    __device__ __forceinline__ explicit Group(int j) : token(j % (kCount / 2)), quad(j / (kCount / 2)) {}
    __device__ __forceinline__ f32x4 join(const Part &part, int waves = kWaves) const {
        const int w = threadIdx.x & 15, at = quad * 16 + token;
        f32x4 v = part[w][at] + part[w][at + Tokens<Few>::kOdd];
        add<0xB1>(v);    // lane ^ 1
        add<0x4E>(v);    // lane ^ 2
        if (waves > 4) add<0x141>(v);    // 7 - lane of 8
        if (waves > 8) add<0x140>(v);    // 15 - lane of 16
        return v;
    }
    template <int Dpp>
    static __device__ __forceinline__ void add(f32x4 &v) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] += __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v[q]), Dpp, 0xf, 0xf, true));
    }
};

// Item (lane % 4) of v.
__device__ __forceinline__ float pick(f32x4 v) {
    const int i = threadIdx.x & 3;
    const float a = i & 1 ? v[1] : v[0], b = i & 1 ? v[3] : v[2];
    return i & 2 ? b : a;
}

// ------------------------------------------------------------------------------------------
// Router
// ------------------------------------------------------------------------------------------

// Sums of 8 experts' logits over the lines first, first + step, ... below `to` by one wave.
template <bool Few>
__device__ __forceinline__ f32x4 logit_sums(const FfnArgs &g, int e0, int first, int step, int to) {
    const Matrix<BSR_WEIGHTS_BF16> m(g.router, nullptr, g.E, g.dim);
    const Expert<BSR_WEIGHTS_BF16> router(m, 0, true);
    const __amdgpu_buffer_rsrc_t x = make_rsrc(g.x, (uint32_t)(g.T * g.dim) * 2u);
    const int token = Tokens<Few>::token();
    const uint32_t row = token < g.T ? (uint32_t)(token * g.dim) * 2u : kPast;
    Sums<Few> acc;
    acc.clear();
    constexpr int B = 4;   // lines in flight
    for (int s0 = first; s0 < to; s0 += B * step) {
        Held w[B];
        bf16x8 v[B][Tokens<Few>::kN];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const int s = s0 + b * step;
            // lines from `to` on: zeros on both sides (an infinite value of x times a zero would be NaN)
            w[b] = Piece8<BSR_WEIGHTS_BF16>(m, s < to ? s : kNoLine).load(m, router, e0);
#pragma unroll
            for (int i = 0; i < Tokens<Few>::kN; ++i) v[b][i] = load_tokens<BSR_WEIGHTS_BF16, Few>(x, s < to ? row : kPast, g.dim, s, 0, i);
        }
#pragma unroll
        for (int b = 0; b < B; ++b) acc.add(expand<BSR_WEIGHTS_BF16>(w[b], 0), v[b]);
    }
    return acc.all();
}

// The joined logits of 8 experts to out[t][E].
template <bool Few>
__device__ __forceinline__ void store_logits(const FfnArgs &g, const Part &part, int e0, float *out) {
    if (threadIdx.x >= Group<Few>::kCount * 16) return;
    const Group<Few> j(threadIdx.x >> 4);
    const float l = pick(j.join(part));
    const int e = e0 + 4 * j.quad + (threadIdx.x & 3);
    if ((threadIdx.x & 15) < 4 && j.token < g.T && e < g.E) out[j.token * g.E + e] = l;
}

// 8 experts and one of `parts` pieces of the columns a work-group.
template <bool Few>
__global__ __launch_bounds__(kThreads) void k_ffn_logits(FfnArgs g) {
    __shared__ Part part;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), e0 = blockIdx.x * 8;
    const int lines = (g.dim + 63) / 64, per = (lines + g.parts - 1) / g.parts, from = blockIdx.y * per;
    part[wave][lane] = logit_sums<Few>(g, e0, from + wave, kWaves, min(from + per, lines));
    __syncthreads();
    store_logits<Few>(g, part, e0, g.logits + (int64_t)blockIdx.y * g.T * g.E);
}

// The experts that some token chose, in ascending order, and each token's slot in them.
struct Chosen {
    int16_t index[kTok * kMaxSlots];
    uint32_t bits[kMaxExperts / 32];
    uint16_t expert[kTok * kMaxSlots];
    uint8_t slot[kTok * kMaxSlots][kTok];   // [chosen expert][token]: its slot there, or kNone
    int count;
};

__device__ __forceinline__ int place_of(const Chosen &c, int e) {   // chosen experts below e
    int n = __popc(c.bits[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < e >> 5; ++w) n += __popc(c.bits[w]);
    return n;
}

// Before anything is chosen; the caller's next barrier publishes it.
__device__ __forceinline__ void clear(const FfnArgs &g, Chosen &c) {
    const int slots = g.T * g.k, i = threadIdx.x;   // slots <= 512 threads
    if (i < (g.E + 31) / 32) c.bits[i] = 0;
    if (i < slots) c.index[i] = -1;
    for (int j = i; j < slots * (kTok / 4); j += kThreads) reinterpret_cast<uint32_t *>(c.slot)[j] = ~0u;
}

__device__ __forceinline__ void choose(Chosen &c, int i, int e) {
    c.index[i] = (int16_t)e;
    atomicOr(&c.bits[e >> 5], 1u << (e & 31));
}

// After a barrier behind the last choose(): the list; the caller's next barrier publishes it.
__device__ __forceinline__ void list(const FfnArgs &g, Chosen &c) {
    const int words = (g.E + 31) / 32, i = threadIdx.x;
    const int e = i < g.T * g.k ? c.index[i] : -1;
    if (i == 0) {
        int n = 0;
        for (int w = 0; w < words; ++w) n += __popc(c.bits[w]);
        c.count = n;
    }
    if (e >= 0) {
        const int a = place_of(c, e);
        c.expert[a] = (uint16_t)e;   // the same value from every slot
        c.slot[a][i / g.k] = (uint8_t)(i % g.k);
    }
}

// Largest of the wave's v.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));   // row rotations by 8, 4, 2, 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

// Router in the work-group: a wave takes a token, lane l its experts l, 64 + l, ...; k rounds of the largest logit, ties to the lowest
// expert (NaN is larger than all, -infinity is never chosen), as bsr_router_fwd. One work-group writes index and weight for the
// down product. (Ranks by counting the better experts of each, 64 comparisons a thread at 16 tokens and 64 experts: 4 us more.)
constexpr int kMostHere = 256;   // experts of a work-group that routes
constexpr int kRounds = kMostHere / 64, kMostParts = 8;

template <bool Few>
__device__ __forceinline__ void route(const FfnArgs &g, Chosen &c, Part &part, float *logit) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (g.route == kAllInOne) {
        for (int e0 = 0; e0 < g.E; e0 += 8) {
            if (e0) __syncthreads();
            part[wave][lane] = logit_sums<Few>(g, e0, wave, kWaves, (g.dim + 63) / 64);
            __syncthreads();
            store_logits<Few>(g, part, e0, logit);
        }
    }
    __syncthreads();
    const int t = wave;   // kTok <= kWaves
    if (t >= g.T) return;
    const __amdgpu_buffer_rsrc_t logits = make_rsrc(g.logits, (uint32_t)(g.parts * g.T * g.E) * 4u);
    float l[kRounds];
    uint32_t key[kRounds];
    int slot[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int e = 64 * r + lane;
        l[r] = -__builtin_inff();
        if (e < g.E) {
            if (g.route == kAllInOne) {
                l[r] = logit[t * g.E + e];
            } else {
                float piece[kMostParts];   // all of them in flight, 0 where there is none
#pragma unroll
                for (int p = 0; p < kMostParts; ++p)
                    piece[p] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                        logits, p < g.parts ? (uint32_t)((p * g.T + t) * g.E + e) * 4u : kPast, 0, 0));
                l[r] = 0.f;
#pragma unroll
                for (int p = 0; p < kMostParts; ++p) l[r] += piece[p];
            }
        }
        const uint32_t bits = __float_as_uint(l[r] + 0.f);   // -0 is 0
        key[r] = bits ^ ((int)bits < 0 ? 0xFFFFFFFFu : 0x80000000u);   // in the order of the values
        if (l[r] != l[r]) key[r] = 0xFFFFFFFFu;
        if (l[r] == -__builtin_inff()) key[r] = 0;
        slot[r] = -1;
    }
    int found = 0;
    float top = 0.f;
    for (; found < g.k; ++found) {
        uint32_t m = key[0];
#pragma unroll
        for (int r = 1; r < kRounds; ++r) m = max(m, key[r]);
        m = wave_max(m);
        if (m == 0) break;
        bool done = false;
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint64_t at = __ballot(key[r] == m);
            if (!done && at) {
                done = true;
                const int who = __builtin_ctzll(at);
                if (found == 0) top = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(l[r]), who));
                if (lane == who) key[r] = 0, slot[r] = found;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (slot[r] >= 0) choose(c, t * g.k + slot[r], 64 * r + lane);
    if (blockIdx.x != 0) return;
    float den = 0.f;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (64 * r + lane < g.E && (slot[r] >= 0 || !g.renorm)) den += __expf(l[r] - top);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) den += __shfl_xor(den, d);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (slot[r] >= 0) {
            g.index[t * g.k + slot[r]] = 64 * r + lane;
            g.weight[t * g.k + slot[r]] = __expf(l[r] - top) / den;
        }
    if (lane >= found && lane < g.k) {
        g.index[t * g.k + lane] = -1;
        g.weight[t * g.k + lane] = 0.f;
    }
}

// ------------------------------------------------------------------------------------------
// h: Q times 8 gate rows and their up rows of one chosen expert a unit; the waves split the columns, Span of them each, and hold
// their tokens' values there over all units. Weights are loaded D units ahead.
// Wide: more columns than the waves hold, taken in several spans whose tokens' values are loaded for every unit.
// Where fewer waves hold the columns, g.waves of them are a set with its own 8 Q rows of a unit: 16 tokens on 64 4-bit experts,
// 1024 / 2048: the layer 86 us, without sets 131 (the down product unsplit); 4 tokens on 64 8-bit ones, 1024 / 1024: 37 | 41.
// ------------------------------------------------------------------------------------------
template <int Form, bool Few, bool Stream, int Span, int Q, int D, bool Wide>
__global__ __launch_bounds__(kThreads) void k_ffn_up(FfnArgs g) {
    using L = Line<Form>;
    constexpr int LN = Span > L::kValues ? Span / L::kValues : 1, N = Tokens<Few>::kN;   // lines a wave
    __shared__ Chosen chosen;
    __shared__ Part part[2][2 * Q];
    __shared__ float logit[kTok * kMostInOne];
    clear(g, chosen);
    if (g.splits > 1 && blockIdx.x == 0)   // (tiles of the down product are fewer than CUs then)
        for (int i = threadIdx.x; i < (g.dim + 7) / 8; i += kThreads) g.done[i] = 0;
    if (g.route == kRouted) {
        __syncthreads();
        const int i = threadIdx.x, e = i < g.T * g.k ? g.index[i] : -1;
        if ((unsigned)e < (unsigned)g.E) choose(chosen, i, e);
        __syncthreads();
    } else {
        route<Few>(g, chosen, part[0][0], logit);
        __syncthreads();
    }
    list(g, chosen);
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), token = Tokens<Few>::token();
    const __amdgpu_buffer_rsrc_t x = make_rsrc(g.x, (uint32_t)(g.T * g.dim) * 2u);
    const uint32_t row = token < g.T ? (uint32_t)(token * g.dim) * 2u : kPast;
    const int waves = Wide ? kWaves : g.waves, set = wave / waves, line = wave % waves, rows = 8 * Q * (kWaves / waves);   // of a unit
    const int tiles = (g.hidden + rows - 1) / rows, count = __builtin_amdgcn_readfirstlane(chosen.count);
    [[maybe_unused]] const int spans = (g.dim + LN * kWaves * L::kValues - 1) / (LN * kWaves * L::kValues);
    const Matrix<Form> m(g.up, g.up_scales, 2 * g.hidden, g.dim);
    bf16x8 v[LN][L::kP][N];
    struct Unit {
        Held w[LN][Q][2];
        uint32_t bias[Q];   // of the row that this thread joins
        int a, n0;          // place of its expert (from count on: none), first gate row
    };
    // groups 2 j and 2 j + 1, neighbours in a wave, join gate and up
    const Group<Few> group(threadIdx.x >> 5);
    const bool gate = !(threadIdx.x & 16), joins = threadIdx.x < 2 * Group<Few>::kCount * 16;
    const int at = 8 * Q * ((threadIdx.x & 15) / waves) + 4 * group.quad + (threadIdx.x & 3);
    // lines of span z: neighbouring ones for neighbouring waves
    auto load_x = [&](int z) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LN; ++i)
#pragma unroll
            for (int p = 0; p < L::kP; ++p)
#pragma unroll
                for (int n = 0; n < N; ++n) v[i][p][n] = load_tokens<Form, Few>(x, row, g.dim, (z * LN + i) * waves + line, p, n);
    };
    auto load_w = [&](Unit &to, int z) __attribute__((always_inline)) {
        const bool live = to.a < count;
        const int e = live ? __builtin_amdgcn_readfirstlane(chosen.expert[live ? to.a : 0]) : 0;
        const Expert<Form> w(m, e, live);
        const __amdgpu_buffer_rsrc_t b = make_rsrc(g.up_bias + (int64_t)e * 2 * g.hidden, g.up_bias ? (uint32_t)g.hidden * 4u : 0u);
        if (z == 0) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
                to.bias[q] = __builtin_amdgcn_raw_buffer_load_b16(b, (uint32_t)(to.n0 + 8 * q + at + (gate ? 0 : g.hidden)) * 2u, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < LN; ++i) {   // (a unit's last rows may lie past the gate's: they are not stored)
            const Piece8<Form> piece(m, (z * LN + i) * waves + line);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                to.w[i][q][0] = piece.template load<Stream>(m, w, to.n0 + 8 * (Q * set + q));
                to.w[i][q][1] = piece.template load<Stream>(m, w, to.n0 + 8 * (Q * set + q) + g.hidden);
            }
        }
    };
    int na = 0, ntile = blockIdx.x;   // of the next unit to load
    auto next = [&](Unit &to) __attribute__((always_inline)) {
        while (ntile >= tiles) ntile -= tiles, ++na;
        to.a = na;
        to.n0 = ntile * rows;
        load_w(to, 0);
        ntile += gridDim.x;
    };
    Sums<Few> acc[Q][2];
    auto products = [&](const Unit &of) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < LN; ++i)
#pragma unroll
            for (int p = 0; p < L::kP; ++p)
#pragma unroll
                for (int q = 0; q < Q; ++q)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[q][c].add(expand<Form>(of.w[i][q][c], p), v[i][p]);
    };
    int turn = 0;
    Unit unit[D];
#pragma unroll
    for (int d = 0; d < D; ++d) next(unit[d]);
    load_x(0);
    for (bool more = true; more;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int a = unit[d].a, n0 = unit[d].n0;
            if (a >= count) {
                more = false;
                break;
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) acc[q][0].clear(), acc[q][1].clear();
            products(unit[d]);
            if constexpr (Wide) {
                for (int z = 1; z < spans; ++z) {
                    load_w(unit[d], z);
                    load_x(z);
                    products(unit[d]);
                }
                load_x(0);
            }
            uint32_t bias[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) bias[q] = unit[d].bias[q];
            next(unit[d]);
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int c = 0; c < 2; ++c) part[turn][2 * q + c][wave][lane] = acc[q][c].all();
            __syncthreads();
            if (joins) {
                const int slot = group.token < g.T ? chosen.slot[a][group.token] : kNone;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float mine = pick(group.join(part[turn][2 * q + !gate], waves)) + from_bf16((uint16_t)bias[q]);
                    const float other = __shfl_xor(mine, 16);
                    const int n = n0 + 8 * q + at;
                    // rounded to bf16: it is an operand of the down product's matrix cores, which in 32 bits would multiply at a 16th
                    // of the rate (the layer's error 0.0024 of its norm, with the result's own rounding alone 0.0017)
                    if (gate && (threadIdx.x & 15) % waves < 4 && slot != kNone && n < g.hidden)
                        g.h[(int64_t)(group.token * g.k + slot) * g.hidden + n] = to_bf16(mine / (1.f + __expf(-mine)) * other);
                }
            }
            turn ^= 1;
        }
    }
}

// ------------------------------------------------------------------------------------------
// out: 8 RS columns a work-group, over all chosen experts; the waves split the lines of all of them, neighbouring ones a wave, so that
// a wave seldom changes its expert.
// Where there are fewer tiles than CUs, g.splits work-groups share the lines of a tile; the last of them to be done adds up the sums of
// all, in the order of their numbers: 8 tokens on 128 experts in bf16, 256 / 1024: the layer 35 us, with one work-group a tile 55; 16
// tokens on 64 4-bit ones, 1024 / 2048: 72 | 84.
// Of 9 to 16 tokens an expert has up to 8 in most calls: then they share an operand as up to 8 tokens of a call do (Packed), column c
// being the expert's c-th token, and its sums go to the tokens' lanes at the expert's end.
// ------------------------------------------------------------------------------------------
template <int Form, bool Few, bool Packed, bool Stream, int RS, int D>
__device__ __forceinline__ void down_sums(const FfnArgs &g, const Chosen &chosen, const float *weight, int n0, int split, f32x4 (&sum)[RS]) {
    using L = Line<Form>;
    constexpr bool Shared = Few || Packed;
    constexpr int N = Tokens<Shared>::kN;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), column = Tokens<Shared>::token();
    const __amdgpu_buffer_rsrc_t h = make_rsrc(g.h, (uint32_t)(g.T * g.k) * (uint32_t)g.hidden * 2u);
    const int steps = (g.hidden + L::kValues - 1) / L::kValues, count = __builtin_amdgcn_readfirstlane(chosen.count);
    const Matrix<Form> m(g.down, g.down_scales, g.dim, g.hidden);

    struct Stage {
        Held w[RS];
        bf16x8 v[L::kP][N];
        int item;           // token k + slot of this lane's column, or -1
        uint32_t tokens;    // Packed: bit t: token t chose the expert
        bool valid, last;   // a line of this wave; its last one of the expert
    };
    // this wave's lines: left of them to load, the next one
    const int total = count * steps, waves = kWaves * g.splits, at = split * kWaves + wave, per = total / waves, more = total % waves;
    int left = per + (at < more ? 1 : 0);
    const int from = at * per + min(at, more);
    int a = from / steps, s = from - a * steps, item = -1;
    uint32_t tokens = 0, row = kPast;
    Expert<Form> w(m, 0, false);
    auto expert = [&]() __attribute__((always_inline)) {   // a's: where its weights and its tokens' rows of h lie
        const bool live = a < count;
        w = Expert<Form>(m, live ? __builtin_amdgcn_readfirstlane(chosen.expert[live ? a : 0]) : 0, live);
        int token = column;
        if constexpr (Packed) {
            tokens = live ? (uint32_t)__ballot(chosen.slot[a][lane & 15] != kNone) & 0xFFFFu : 0u;
            uint32_t rest = tokens;
#pragma unroll
            for (int i = 0; i < 7; ++i) rest = i < column ? rest & (rest - 1) : rest;
            token = rest ? __builtin_ctz(rest) : -1;
        }
        const int slot = live && token >= 0 ? chosen.slot[a][token] : kNone;
        item = slot != kNone ? token * g.k + slot : -1;
        row = item >= 0 ? (uint32_t)item * (uint32_t)g.hidden * 2u : kPast;
    };
    auto load = [&](Stage &st) __attribute__((always_inline)) {
        if (s == steps) {
            s = 0;
            ++a;
            expert();
        }
        st.valid = left > 0;
        st.last = left == 1 || s + 1 == steps;
        st.item = item;
        st.tokens = tokens;
        const Piece8<Form> piece(m, left > 0 ? s : kNoLine);
#pragma unroll
        for (int i = 0; i < RS; ++i) st.w[i] = piece.template load<Stream>(m, w, n0 + 8 * i);
#pragma unroll
        for (int p = 0; p < L::kP; ++p)
#pragma unroll
            for (int n = 0; n < N; ++n) st.v[p][n] = load_tokens<Form, Shared>(h, left > 0 ? row : kPast, g.hidden, s, p, n);
        ++s;
        --left;
    };
    Sums<Shared> acc[RS];
#pragma unroll
    for (int i = 0; i < RS; ++i) acc[i].clear();
    Stage st[D];
    expert();
#pragma unroll
    for (int d = 0; d < D; ++d) load(st[d]);
    for (bool go = true; go;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (!st[d].valid) {
                go = false;
                break;
            }
#pragma unroll
            for (int p = 0; p < L::kP; ++p)
#pragma unroll
                for (int i = 0; i < RS; ++i) acc[i].add(expand<Form>(st[d].w[i], p), st[d].v[p]);
            // the expert's last line of this wave: its sums, weighted, go into the tokens that chose it (others' are dropped: infinite
            // weights times no value)
            if (st[d].last) {
                const float by = weight[max(st[d].item, 0)];
                const int t = lane & 15;
                const bool mine = Packed ? lane < 32 && (st[d].tokens >> t & 1) : st[d].item >= 0;
                const int even = 4 * ((lane & 16) + __popc(st[d].tokens & ((1u << t) - 1u))), odd = even + 4 * Tokens<true>::kOdd;
#pragma unroll
                for (int i = 0; i < RS; ++i) {
                    const f32x4 v = acc[i].all();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float one = v[q] * by;
                        if constexpr (Packed)
                            one = __int_as_float(__builtin_amdgcn_ds_bpermute(even, __float_as_int(one))) +
                                  __int_as_float(__builtin_amdgcn_ds_bpermute(odd, __float_as_int(one)));
                        sum[i][q] = mine ? sum[i][q] + one : sum[i][q];
                    }
                    acc[i].clear();
                }
            }
            load(st[d]);
        }
    }
}

template <int Form, bool Few, bool Stream, int RS>
__global__ __launch_bounds__(kThreads) void k_ffn_down(FfnArgs g) {
    __shared__ Chosen chosen;
    __shared__ Part part[RS];
    __shared__ float weight[kTok * kMaxSlots];
    clear(g, chosen);
    __syncthreads();
    if ((int)threadIdx.x < g.T * g.k) {
        const int e = g.index[threadIdx.x];
        weight[threadIdx.x] = g.weight[threadIdx.x];
        if ((unsigned)e < (unsigned)g.E) choose(chosen, threadIdx.x, e);
    }
    __syncthreads();
    list(g, chosen);
    __syncthreads();
    __shared__ bool last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = blockIdx.x * 8 * RS, split = blockIdx.y;
    f32x4 sum[RS] = {};
    // Lines loaded ahead. More than three, which the registers could hold for most, win nothing, and of 4-bit weights the third cannot pay
    // for its code, fetched cold in every launch: 4 tokens, 4096 / 7168 67 us | 70, 16 tokens on 32 experts, 2048 / 2048 68 | 69.
    constexpr int D = Form == BSR_WEIGHTS_MX4 ? 2 : 3;
    if constexpr (Few) {
        down_sums<Form, true, false, Stream, RS, D>(g, chosen, weight, n0, split, sum);
    } else {
        bool many = false;   // an expert with more than 8 tokens
        for (int a = lane; a < chosen.count; a += 64) {
            int none = 0;
#pragma unroll
            for (int i = 0; i < kTok / 4; ++i) none += __popc(reinterpret_cast<const uint32_t *>(chosen.slot[a])[i] & 0x80808080u);
            many |= kTok - none > 8;
        }
        if (__ballot(many)) down_sums<Form, false, false, Stream, RS, 2>(g, chosen, weight, n0, split, sum);
        else down_sums<Form, false, true, Stream, RS, D>(g, chosen, weight, n0, split, sum);
    }
#pragma unroll
    for (int i = 0; i < RS; ++i) part[i][wave][lane] = sum[i];
    __syncthreads();
    const Group<Few> j((threadIdx.x >> 4) % Group<Few>::kCount);
    const int set = (threadIdx.x >> 4) / Group<Few>::kCount, t = j.token, n = n0 + 8 * set + 4 * j.quad + (threadIdx.x & 3);
    const bool mine = threadIdx.x < RS * Group<Few>::kCount * 16 && (threadIdx.x & 15) < 4 && t < g.T && n < g.dim;
    float v = 0.f;
    if (threadIdx.x < RS * Group<Few>::kCount * 16) v = pick(j.join(part[set]));
    if (g.splits > 1) {
        // Stores and loads that go past the XCDs' own caches, and a wait until the stores have arrived, in place of fences, which write
        // the caches back: those took 80 us.
        float *at = g.partial + (int64_t)t * g.dim + n;
        const int64_t next = (int64_t)g.T * g.dim;
        if (mine) __hip_atomic_store(at + split * next, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(&g.done[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)g.splits - 1;
        __syncthreads();
        if (!last) return;
        v = 0.f;
        if (mine)
            for (int i = 0; i < g.splits; ++i) v += __hip_atomic_load(at + i * next, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (mine) {
        if (g.down_bias)
            for (int i = 0; i < g.k; ++i) {
                const int e = chosen.index[t * g.k + i];
                if (e >= 0) v = fmaf(weight[t * g.k + i], from_bf16(g.down_bias[(int64_t)e * g.dim + n]), v);
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

// Who finds the experts of a call. kAllInOne | kFromLogits, us: one token on 8 bf16 experts, 2048 / 1024: 15.8 | 17.6, on 16 8-bit ones,
// 1024 / 1024: 16.4 | 18.0, 24: 17.3 | 17.5; 4 tokens on 32, 1024 / 2048: 36 | 31.6; on 8 with 4096 columns 66.2 | 66.1, 16: 23.0 | 20.6. The router's kernel
// instead of kFromLogits: 8 tokens on 64 8-bit experts, 2048 / 1024: 48.7 | 46.7; more than 256 experts do not fit its registers.
Route route_of(int E, int64_t dim) {
    if (E > kMostHere) return kRouted;
    return E <= kMostInOne && E * dim <= 32768 ? kAllInOne : kFromLogits;
}

// Pieces of the logits' sums: 8 lines each, half a line a wave.
int parts_of(Route r, int dim) { return r == kFromLogits ? std::min(kMostParts, (dim + 511) / 512) : 1; }

template <int Form, bool Few, bool Stream>
void launch_up(const FfnArgs &g, const FfnVariant &v, hipStream_t st) {
    const int rows = 8 * v.q * (kWaves / v.waves);
    const int64_t units = (int64_t)std::min(g.E, g.T * g.k) * ((g.hidden + rows - 1) / rows);
    auto up = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(units, kCUs)), dim3(kThreads), 0, st, g);
    };
    // units loaded ahead: what the registers hold beside the tokens' values
    constexpr int UD = Form == BSR_WEIGHTS_BF16 ? 1 : Form == BSR_WEIGHTS_FP8 ? 2 : 3;
    constexpr int QD = Form == BSR_WEIGHTS_BF16 || (Form == BSR_WEIGHTS_MX4 && !Few) ? 1 : 2;
    if (v.wide) up(k_ffn_up<Form, Few, Stream, 128, 1, 1, true>);
    else if (v.q == 2) up(k_ffn_up<Form, Few, Stream, 128, 2, QD, false>);
    else up(k_ffn_up<Form, Few, Stream, 256, 1, UD, false>);
}

template <int Form, bool Few, bool Stream>
void launch_down(const FfnArgs &g, const FfnVariant &v, hipStream_t st) {
    const dim3 grid((unsigned)((g.dim + 8 * v.rs - 1) / (8 * v.rs)), (unsigned)v.splits);
    if (v.rs == 2) hipLaunchKernelGGL((k_ffn_down<Form, Few, Stream, 2>), grid, dim3(kThreads), 0, st, g);
    else hipLaunchKernelGGL((k_ffn_down<Form, Few, Stream, 1>), grid, dim3(kThreads), 0, st, g);
}

template <int Form, bool Few>
void launch_products(const FfnArgs &g, const FfnVariant &v, hipStream_t st) {
    if (v.stream_up) launch_up<Form, Few, true>(g, v, st);
    else launch_up<Form, Few, false>(g, v, st);
    if (v.stream_down) launch_down<Form, Few, true>(g, v, st);
    else launch_down<Form, Few, false>(g, v, st);
}

template <int Form>
void launch_products(FfnArgs g, hipStream_t st) {
    const FfnVariant v = ffn_variant(Line<Form>::kValues, g.T, g.dim, g.hidden, g.E, g.k);
    g.waves = v.waves;
    g.splits = v.splits;
    if (v.few) launch_products<Form, true>(g, v, st);
    else launch_products<Form, false>(g, v, st);
}

}  // namespace

size_t expert_ffn_workspace_bytes(int T, int dim, int hidden, int E, int k) {
    const size_t splits = ffn_variant(Line<BSR_WEIGHTS_BF16>::kValues, T, dim, hidden, E, k).splits;   // the most of all forms
    return up16((size_t)parts_of(route_of(E, dim), dim) * T * E * 4) + 2 * up16((size_t)T * k * 4) + up16((size_t)T * k * hidden * 2) +
           (splits > 1 ? up16((size_t)dim / 8 * 4) + splits * T * dim * 4 : 0);
}

int32_t launch_expert_ffn(const uint16_t *x, int T, int dim, int hidden, int E, int k, bool renorm, const uint16_t *router,
                          int form, const void *up, const uint8_t *up_scales, const void *down, const uint8_t *down_scales,
                          const uint16_t *up_bias, const uint16_t *down_bias, uint16_t *out, void *workspace, void *stream) {
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const Route r = route_of(E, dim);
    FfnArgs g{x, T, dim, hidden, E, k, renorm, r, parts_of(r, dim), kWaves, router, up, down, up_scales, down_scales, up_bias, down_bias, out,
              nullptr, nullptr, nullptr, nullptr, 1, nullptr, nullptr};
    g.logits = reinterpret_cast<float *>(ws);
    ws += up16((size_t)g.parts * T * E * 4);
    g.index = reinterpret_cast<int32_t *>(ws);
    ws += up16((size_t)T * k * 4);
    g.weight = reinterpret_cast<float *>(ws);
    ws += up16((size_t)T * k * 4);
    g.h = reinterpret_cast<uint16_t *>(ws);
    ws += up16((size_t)T * k * hidden * 2);
    g.done = reinterpret_cast<uint32_t *>(ws);
    g.partial = reinterpret_cast<float *>(ws + up16((size_t)dim / 8 * 4));
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (r != kAllInOne) {
        const dim3 grid((unsigned)((E + 7) / 8), (unsigned)g.parts);
        if (T <= 8) hipLaunchKernelGGL(k_ffn_logits<true>, grid, dim3(kThreads), 0, st, g);
        else hipLaunchKernelGGL(k_ffn_logits<false>, grid, dim3(kThreads), 0, st, g);
    }
    if (r == kRouted)
        if (const int32_t bad = launch_router_fwd(g.logits, BSR_LOGITS_F32, T, E, k, renorm, g.index, g.weight, stream)) return bad;
    if (form == BSR_WEIGHTS_BF16) launch_products<BSR_WEIGHTS_BF16>(g, st);
    else if (form == BSR_WEIGHTS_MX4) launch_products<BSR_WEIGHTS_MX4>(g, st);
    else launch_products<BSR_WEIGHTS_FP8>(g, st);
    return launched("bsr_expert_ffn");
}

}  // namespace bsr
