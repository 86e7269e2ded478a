// bsr_experts.hip -- the router, the plan and the sum of an expert layer (include/bsr_experts.h).
//
// All of these are bound by the bytes they read and write, or, for a few tokens, by the launch (2.9 us on the host;
// the kernels then take 3 to 4 us). Times below are kernel times on one MI355X, inputs not in the caches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "bsr_device.hpp"
#include "bsr_experts_internal.hpp"

namespace bsr {
namespace {

using namespace dev;

constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load_logit(const float *p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t *p) { return from_bf16(*p); }
__device__ __forceinline__ void store_logit(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t *p, float v) { *p = to_bf16(v); }

// An unsigned key in the order of the values: -infinity is the smallest (key 0x007FFFFF), both zeros are
// equal, NaN of either sign is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);   // -0 + 0 = +0
    if ((b & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The value behind a key (NaN for the largest key).
__device__ __forceinline__ float key_value(uint32_t key) {
    return key == 0xFFFFFFFFu ? __builtin_nanf("") : __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

// Rotation by D lanes within each row of 16 lanes, on the vector units (no LDS crossbar).
template <int D>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + D, 0xF, 0xF, true);
}
// Maximum and sum over each group of G = 16 or 64 lanes.
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    v = max(v, row_rotate<8>(v));
    v = max(v, row_rotate<4>(v));
    v = max(v, row_rotate<2>(v));
    v = max(v, row_rotate<1>(v));
    if constexpr (G == 64) {
        v = max(v, (uint32_t)__shfl_xor((int)v, 16));
        v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
    v += __uint_as_float(row_rotate<8>(__float_as_uint(v)));
    v += __uint_as_float(row_rotate<4>(__float_as_uint(v)));
    v += __uint_as_float(row_rotate<2>(__float_as_uint(v)));
    v += __uint_as_float(row_rotate<1>(__float_as_uint(v)));
    if constexpr (G == 64) {
        v += __shfl_xor(v, 16);
        v += __shfl_xor(v, 32);
    }
    return v;
}

// The NV logits of experts first .. first + NV - 1 (-infinity past E). whole: rows are whole 16-byte pieces.
template <typename L, int NV>
__device__ __forceinline__ void load_logits(const L *row, int first, int E, bool whole, float *v) {
    constexpr int kPiece = 16 / sizeof(L);
    if constexpr (NV % kPiece == 0) {
        if (whole) {
#pragma unroll
            for (int p = 0; p < NV / kPiece; ++p) {
                u32x4 w = {0, 0, 0, 0};
                const bool in = first + p * kPiece < E;
                if (in) w = *reinterpret_cast<const u32x4 *>(row + first + p * kPiece);
#pragma unroll
                for (int i = 0; i < kPiece; ++i) {
                    const uint32_t word = w[i * sizeof(L) / 4];
                    const float f = sizeof(L) == 4 ? __uint_as_float(word) : __uint_as_float((i & 1) ? word & 0xFFFF0000u : word << 16);
                    v[p * kPiece + i] = in ? f : kNegInf;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = first + i < E ? load_logit(row + first + i) : kNegInf;
}

// Router forward: a token takes a group of G lanes, lane l the experts l NV .. l NV + NV - 1. k rounds: the
// largest key of the group, then the lowest lane and expert that holds it (ties to the lowest expert); a taken key
// becomes 0, below every logit's. Slot j stays with lane j until the end. 16 lanes a token (up to 256 experts and
// 16 slots) keep the rounds on row rotations: 16390 x 128 bf16, k = 8 takes 7.5 us (a wave a token with
// shuffles: 21); its bytes would take 1, the k dependent rounds bound it.
template <typename L, int NV, int G>
__global__ __launch_bounds__(256) void k_router_fwd(const L *__restrict__ logits, int T, int E, int k, int renorm,
                                                    bool whole, int32_t *__restrict__ index, float *__restrict__ weight) {
    const int lane = threadIdx.x & 63, gl = lane & (G - 1), g0 = lane & ~(G - 1);
    const int t = blockIdx.x * (256 / G) + threadIdx.x / G;
    const bool in = t < T;
    float v[NV];
    uint32_t key[NV];
    load_logits<L, NV>(logits + (int64_t)min(t, T - 1) * E, gl * NV, E, whole, v);
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = gl * NV + i < E ? order_key(v[i]) : 0;
    uint32_t top = 0, mine = 0;
    int pick = -1;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = max(best, key[i]);
        const uint32_t all = group_max<G>(best);
        const bool some = all > kKeyNegInf;   // else nothing but -infinity is left
        const uint64_t have = __ballot(best == all) >> g0;
        const int owner = __builtin_ctzll(have);
        int at = -1;
        if (some && gl == owner) {
#pragma unroll
            for (int i = NV - 1; i >= 0; --i) at = key[i] == all ? i : at;
#pragma unroll
            for (int i = 0; i < NV; ++i) key[i] = i == at ? 0 : key[i];
        }
        const int e = __shfl(at, g0 + owner) + owner * NV;
        if (j == 0) top = all;
        if (some && gl == j) {
            pick = e;
            mine = all;
        }
    }
    // Weights in 32 bits. top is a real logit, +infinity or NaN whenever any slot was filled.
    const float m = top > kKeyNegInf ? key_value(top) : 0.f;
    const float ex = pick >= 0 ? expf(key_value(mine) - m) : 0.f;
    float den = ex;
    if (!renorm) {
        den = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) den += expf(v[i] - m);   // -infinity gives 0
    }
    den = group_sum<G>(den);
    if (in && gl < k) {
        index[(int64_t)t * k + gl] = pick;
        weight[(int64_t)t * k + gl] = pick >= 0 ? ex / den : 0.f;
    }
}

// Router backward, the same lanes. Not renormalised: p is computed again from the logits (reading them costs less than
// storing p would). 16390 x 128 bf16: 6.3 us.
template <typename L, int NV, int G>
__global__ __launch_bounds__(256) void k_router_bwd(const L *__restrict__ logits, int T, int E, int k, int renorm,
                                                    bool whole, const int32_t *__restrict__ index,
                                                    const float *__restrict__ weight, const float *__restrict__ dweight,
                                                    L *__restrict__ dlogits) {
    const int lane = threadIdx.x & 63, gl = lane & (G - 1), g0 = lane & ~(G - 1);
    const int t = blockIdx.x * (256 / G) + threadIdx.x / G;
    const bool in = t < T;
    int pick = -1;
    float w = 0.f, g = 0.f;
    if (in && gl < k) {
        pick = index[(int64_t)t * k + gl];
        if ((unsigned)pick < (unsigned)E) {
            w = weight[(int64_t)t * k + gl];
            g = dweight[(int64_t)t * k + gl];
        } else {
            pick = -1;
        }
    }
    const float inner = group_sum<G>(w * g);
    float v[NV], d[NV];
    if (!renorm) {
        load_logits<L, NV>(logits + (int64_t)min(t, T - 1) * E, gl * NV, E, whole, v);
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) best = max(best, gl * NV + i < E ? order_key(v[i]) : 0u);
        const uint32_t top = group_max<G>(best);
        const bool none = top <= kKeyNegInf;
        const float m = none ? 0.f : key_value(top);
        float den = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = expf(v[i] - m);
            den += v[i];
        }
        den = group_sum<G>(den);
        const float scale = none ? 0.f : inner / den;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = -v[i] * scale;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = 0.f;
    }
    const float add = renorm ? w * (g - inner) : w * g;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl(pick, g0 + j) - gl * NV;
        const float a = __shfl(add, g0 + j);
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] += e == i ? a : 0.f;
    }
    if (!in) return;
    L *out = dlogits + (int64_t)t * E + gl * NV;
    constexpr int kPiece = 16 / sizeof(L);
    if constexpr (NV % kPiece == 0) {
        if (whole) {
#pragma unroll
            for (int p = 0; p < NV / kPiece; ++p) {
                if (gl * NV + p * kPiece >= E) break;
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *f = d + p * kPiece;
                    o[i] = sizeof(L) == 4 ? __float_as_uint(f[i])
                                          : (uint32_t)to_bf16(f[(2 * i) % kPiece]) | ((uint32_t)to_bf16(f[(2 * i + 1) % kPiece]) << 16);
                }
                *reinterpret_cast<u32x4 *>(out + p * kPiece) = o;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (gl * NV + i < E) store_logit(out + i, d[i]);
}

// ------------------------------------------------------------------------------------------
// The plan: a stable counting sort of S = T k slots by expert.
// A slot's row is offsets[e] + the slots of e in earlier chunks + those in earlier rounds of 1024 slots of its
// chunk + those in earlier waves of the round + those in lower lanes of its wave (a ballot for each bit of e).
// Up to 1024 slots, one work-group does everything. Beyond that one launch counts each chunk's slots, and in
// a second one every chunk adds up the counts that it needs by itself; chunks have as many rounds as keep
// their number within 256, so that this stays a few loads a thread. 131120 slots, 128 experts: 2.6 + 6.6 us (three launches,
// the middle one a single work-group that walked the counts: 30 us).
// ------------------------------------------------------------------------------------------
constexpr int kPlanRound = BSR_EXPERT_PLAN_SLOTS, kPlanChunks = 256;

// Counts of this round's waves in cnt[16][E] (16-bit) and this slot's rank among its wave's.
__device__ __forceinline__ int plan_rank(int e, int E, int bits, uint16_t *cnt) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    uint64_t same = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const bool set = (e >> b) & 1;
        const uint64_t m = __ballot(set);
        same &= set ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (e < E && rank == 0) cnt[wave * E + e] = (uint16_t)__popcll(same);
    return rank;
}

__device__ __forceinline__ int plan_expert(const int32_t *index, int64_t s, int64_t S, int E) {
    const int e = s < S ? index[s] : -1;
    return (unsigned)e < (unsigned)E ? e : E;
}

// Exclusive prefix over the block's 1024 threads of one value each; *total = the sum.
__device__ __forceinline__ int block_prefix(int v, int *scratch, int *total) {
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    int x = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(x, d);
        if (lane >= d) x += o;
    }
    if (lane == 63) scratch[wave] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        const int c = scratch[w];
        before += w < wave ? c : 0;
        all += c;
    }
    *total = all;
    return before + x - v;
}

__global__ __launch_bounds__(kPlanRound) void k_plan_count(const int32_t *__restrict__ index, int64_t S, int E, int rounds,
                                                           int32_t *__restrict__ counts) {
    __shared__ int hist[kMaxExperts];
    const int tid = threadIdx.x;
    for (int i = tid; i < E; i += kPlanRound) hist[i] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * rounds * kPlanRound;
    for (int r = 0; r < rounds; ++r) {
        const int e = plan_expert(index, s0 + (int64_t)r * kPlanRound + tid, S, E);
        if (e < E) atomicAdd(&hist[e], 1);   // whole numbers: the order does not matter
    }
    __syncthreads();
    for (int i = tid; i < E; i += kPlanRound) counts[(int64_t)blockIdx.x * E + i] = hist[i];
}

// counts: [chunks][E], or NULL for a single chunk of one round.
__global__ __launch_bounds__(kPlanRound) void k_plan_write(const int32_t *__restrict__ index, int64_t S, int k, int E,
                                                           int bits, int rounds, int chunks,
                                                           const int32_t *__restrict__ counts,
                                                           int32_t *__restrict__ offsets, int32_t *__restrict__ row_token,
                                                           int32_t *__restrict__ slot_row) {
    extern __shared__ uint16_t cnt[];   // [16][E]
    __shared__ int scratch[16];
    __shared__ int first[kMaxExperts], all[kMaxExperts];   // next row of each expert in this chunk; its slots
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < 16 * E; i += kPlanRound) cnt[i] = 0;
    int before_chunk = 0, mine = 0;
    int e = 0, rank = 0;
    if (counts) {
        if (tid < E) first[tid] = all[tid] = 0;
        __syncthreads();
        // thread (part, expert): every parts-th chunk
        const int parts = kPlanRound / E, part = tid / E, ex = tid - part * E;
        if (part < parts) {
            int b = 0, a = 0;
#pragma unroll 8
            for (int c = part; c < chunks; c += parts) {
                const int n = counts[(int64_t)c * E + ex];
                a += n;
                b += c < (int)blockIdx.x ? n : 0;
            }
            atomicAdd(&all[ex], a);
            atomicAdd(&first[ex], b);
        }
        __syncthreads();
        if (tid < E) {
            mine = all[tid];
            before_chunk = first[tid];
        }
    } else {
        __syncthreads();
        e = plan_expert(index, tid, S, E);
        rank = plan_rank(e, E, bits, cnt);
        __syncthreads();
        if (tid < E)
            for (int w = 0; w < 16; ++w) mine += cnt[w * E + tid];
    }
    int live;
    const int before = block_prefix(mine, scratch, &live);
    if (tid < E) {
        first[tid] = before + before_chunk;
        if (blockIdx.x == 0) offsets[tid] = before;
    }
    if (tid == 0 && blockIdx.x == 0) offsets[E] = live;
    __syncthreads();
    for (int r = 0; r < rounds; ++r) {
        const int64_t s = ((int64_t)blockIdx.x * rounds + r) * kPlanRound + tid;
        if (counts) {
            e = plan_expert(index, s, S, E);
            rank = plan_rank(e, E, bits, cnt);
            __syncthreads();
        }
        int row = -1;
        if (e < E) {
            row = first[e] + rank;
            for (int w = 0; w < wave; ++w) row += cnt[w * E + e];
        }
        if (s < S) {
            slot_row[s] = row;
            if (row >= 0) row_token[row] = (int32_t)(s / k);
            if (s >= live) row_token[s] = -1;
        }
        if (r + 1 < rounds) {
            __syncthreads();
            if (tid < E)
                for (int w = 0; w < 16; ++w) {
                    first[tid] += cnt[w * E + tid];
                    cnt[w * E + tid] = 0;
                }
            __syncthreads();
        }
    }
}

// ------------------------------------------------------------------------------------------
// The sum over a token's rows and its gradient: 8 columns a thread, so that a wave takes 1 KB of a row. 8191 tokens, k = 8,
// N = 2048: forward 55 us (302 MB, 5.5 TB/s; 76 us behind other work, with nothing of Y in the last-level cache), backward, one
// wave a slot, 113 us (570 MB, 5.0 TB/s; 100 behind the forward, which leaves Y there).
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void unpack8(u32x4 v, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ u32x4 pack8(const float *f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)to_bf16(f[2 * i]) | ((uint32_t)to_bf16(f[2 * i + 1]) << 16);
    return v;
}

// One wave takes 512 columns of a token, so that its rows and weights are scalars; a row behind a descriptor of its own,
// of no bytes where the slot has no row: that load reads zeros without a branch, and Rows rows are in flight. The waves of a
// row follow one another (with all first pieces first: 70 us instead of 55). Rows covers k up to 8; 8 of them
// for k = 2 (16384 tokens, N = 4096): 78 us instead of 74.
constexpr int kCombineTokens = 1 << 14;   // tokens of one slice of the grid (blockIdx.y): its threads fit 32 bits for every N

template <int Rows>
__global__ __launch_bounds__(256) void k_combine_fwd(const uint16_t *__restrict__ Y, int T, int k, int N, int R,
                                                     const int32_t *__restrict__ slot_row,
                                                     const float *__restrict__ weight, uint16_t *__restrict__ out,
                                                     uint32_t pieces) {
    const uint32_t id = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = (int)blockIdx.y * kCombineTokens + (int)(id / pieces);
    const int c = (int)(id % pieces) * 512 + (int)(threadIdx.x & 63) * 8;
    if (t >= T) return;
    const int64_t s0 = (int64_t)t * k;
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += Rows) {
        // lane j % Rows looks at slot j0 + j
        const int64_t s = s0 + min(j0 + (int)(threadIdx.x & (Rows - 1)), k - 1);
        const int r = slot_row[s];
        const float wr = weight ? weight[s] : 1.f;
        const bool there = j0 + (int)(threadIdx.x & (Rows - 1)) < k && (unsigned)r < (unsigned)R;
        const int rows = there ? r : -1;
        const float ws = there ? wr : 0.f;
        u32x4 y[Rows];
#pragma unroll
        for (int j = 0; j < Rows; ++j) {
            const int row = __builtin_amdgcn_readlane(rows, j);
            y[j] = __builtin_amdgcn_raw_buffer_load_b128(make_rsrc(Y + (int64_t)max(row, 0) * N, row < 0 ? 0u : (uint32_t)N * 2u),
                                                         (uint32_t)c * 2u, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < Rows; ++j) {
            const float w = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(ws), j));
            float f[8];
            unpack8(y[j], f);
#pragma unroll
            for (int v = 0; v < 8; ++v) acc[v] += w * f[v];
        }
    }
    if (c < N) *reinterpret_cast<u32x4 *>(out + (int64_t)t * N + c) = pack8(acc);
}

__global__ __launch_bounds__(256) void k_combine_bwd(const uint16_t *__restrict__ dout, const uint16_t *__restrict__ Y,
                                                     int k, int E, int N, int R, const int32_t *__restrict__ offsets,
                                                     const int32_t *__restrict__ slot_row,
                                                     const float *__restrict__ weight, uint16_t *__restrict__ dY,
                                                     float *__restrict__ dweight) {
    const int lane = threadIdx.x & 63, s = blockIdx.x * 4 + (threadIdx.x >> 6);   // one wave a slot
    if (s >= R) return;
    const int n8 = N >> 3;
    const int row = slot_row[s];
    float dot = 0.f;
    if ((unsigned)row < (unsigned)R) {
        const float w = weight ? weight[s] : 1.f;
        const uint16_t *d = dout + (int64_t)(s / k) * N, *y = Y + (int64_t)row * N;
        for (int c = lane; c < n8; c += 64) {
            float a[8], b[8];
            unpack8(*reinterpret_cast<const u32x4 *>(d + c * 8), a);
            unpack8(*reinterpret_cast<const u32x4 *>(y + c * 8), b);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                dot += a[v] * b[v];
                a[v] *= w;
            }
            *reinterpret_cast<u32x4 *>(dY + (int64_t)row * N + c * 8) = pack8(a);
        }
        dot = wave_sum(dot);
    }
    if (lane == 0) dweight[s] = dot;
    if (s >= offsets[E])   // row s belongs to no slot
        for (int c = lane; c < n8; c += 64) *reinterpret_cast<u32x4 *>(dY + (int64_t)s * N + c * 8) = u32x4{0, 0, 0, 0};
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

int bits_for(int E) {   // bits that tell 0 .. E apart
    int b = 1;
    while ((1 << b) <= E) ++b;
    return b;
}

template <typename L>
int32_t router(bool fwd, const void *logits, int T, int E, int k, bool renorm, int32_t *index, float *weight,
               const float *dweight, void *dlogits, hipStream_t st) {
    const L *lg = static_cast<const L *>(logits);
    const bool whole = (int64_t)E * sizeof(L) % 16 == 0;
    auto run = [&](auto nv, auto group) {
        constexpr int NV = decltype(nv)::value, G = decltype(group)::value;
        const dim3 grid((unsigned)((T + 256 / G - 1) / (256 / G))), block(256);
        if (fwd)
            hipLaunchKernelGGL((k_router_fwd<L, NV, G>), grid, block, 0, st, lg, T, E, k, (int)renorm, whole, index, weight);
        else
            hipLaunchKernelGGL((k_router_bwd<L, NV, G>), grid, block, 0, st, lg, T, E, k, (int)renorm, whole, index, weight,
                               dweight, static_cast<L *>(dlogits));
    };
    using std::integral_constant;
    if (E > 256) run(integral_constant<int, 16>{}, integral_constant<int, 64>{});
    else if (k > 16) run(integral_constant<int, 4>{}, integral_constant<int, 64>{});
    else if (E <= 64) run(integral_constant<int, 4>{}, integral_constant<int, 16>{});
    else if (E <= 128) run(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    else run(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    return launched(fwd ? "bsr_router_fwd" : "bsr_router_bwd");
}

}  // namespace

int32_t launch_router_fwd(const void *logits, int32_t type, int T, int E, int k, bool renorm, int32_t *index,
                          float *weight, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return type == BSR_LOGITS_F32
               ? router<float>(true, logits, T, E, k, renorm, index, weight, nullptr, nullptr, st)
               : router<uint16_t>(true, logits, T, E, k, renorm, index, weight, nullptr, nullptr, st);
}

int32_t launch_router_bwd(const void *logits, int32_t type, int T, int E, int k, bool renorm, const int32_t *index,
                          const float *weight, const float *dweight, void *dlogits, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    int32_t *ix = const_cast<int32_t *>(index);
    float *w = const_cast<float *>(weight);
    return type == BSR_LOGITS_F32 ? router<float>(false, logits, T, E, k, renorm, ix, w, dweight, dlogits, st)
                                  : router<uint16_t>(false, logits, T, E, k, renorm, ix, w, dweight, dlogits, st);
}

static int plan_rounds(int64_t slots) { return (int)((slots + kPlanRound * kPlanChunks - 1) / (kPlanRound * kPlanChunks)); }

size_t expert_plan_workspace_bytes(int64_t slots, int E) {
    if (slots <= kPlanRound) return 0;
    const int64_t chunk = (int64_t)plan_rounds(slots) * kPlanRound;
    return (size_t)((slots + chunk - 1) / chunk) * E * sizeof(int32_t);
}

int32_t launch_expert_plan(const int32_t *index, int T, int k, int E, int32_t *offsets, int32_t *row_token,
                           int32_t *slot_row, void *workspace, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t S = (int64_t)T * k;
    const int bits = bits_for(E), rounds = std::max(1, plan_rounds(S));
    const int chunks = std::max<int>(1, (int)((S + rounds * kPlanRound - 1) / (rounds * kPlanRound)));
    const size_t lds = 16 * (size_t)E * sizeof(uint16_t);
    int32_t *counts = S <= kPlanRound ? nullptr : static_cast<int32_t *>(workspace);
    if (counts)
        hipLaunchKernelGGL(k_plan_count, dim3(chunks), dim3(kPlanRound), 0, st, index, S, E, rounds, counts);
    hipLaunchKernelGGL(k_plan_write, dim3(chunks), dim3(kPlanRound), lds, st, index, S, k, E, bits, rounds, chunks, counts,
                       offsets, row_token, slot_row);
    return launched("bsr_expert_plan");
}

int32_t launch_combine_fwd(const uint16_t *Y, int T, int k, int N, const int32_t *slot_row, const float *weight,
                           uint16_t *out, void *stream) {
    // as many outputs of 8 columns as the other operators' grids hold, whatever the pieces of a row round up to
    if (const int32_t bad = check_grid(((int64_t)T * (N / 8) + 255) / 256, 256, "bsr_expert_combine_fwd")) return bad;
    const int pieces = (N + 511) / 512;
    const dim3 grid((unsigned)((std::min(T, kCombineTokens) * pieces + 3) / 4),
                    (unsigned)((T + kCombineTokens - 1) / kCombineTokens));
    hipLaunchKernelGGL(k <= 2 ? k_combine_fwd<2> : k <= 4 ? k_combine_fwd<4> : k_combine_fwd<8>, grid, dim3(256), 0,
                       static_cast<hipStream_t>(stream), Y, T, k, N, T * k, slot_row, weight, out,
                       (uint32_t)pieces);
    return launched("bsr_expert_combine_fwd");
}

int32_t launch_combine_bwd(const uint16_t *dout, const uint16_t *Y, int T, int k, int E, int N, const int32_t *offsets,
                           const int32_t *slot_row, const float *weight, uint16_t *dY, float *dweight, void *stream) {
    const int R = T * k;
    hipLaunchKernelGGL(k_combine_bwd, dim3((unsigned)((R + 3) / 4)), dim3(256), 0, static_cast<hipStream_t>(stream),
                       dout, Y, k, E, N, R, offsets, slot_row, weight, dY, dweight);
    return launched("bsr_expert_combine_bwd");
}

}  // namespace bsr
