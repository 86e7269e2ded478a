// bsr_experts.hip -- the router, the plan and the sum of an expert layer (include/bsr_experts.h).
//
// All of these are bound by the bytes they read and write, or, for a few tokens, by one launch.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <string>

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

// Router forward, one wave a token: lane l holds the logits of experts l + 64 i. k rounds of a wave-wide
// maximum over (key, lowest expert); a taken expert's key becomes 0, below every logit's.
template <typename L, int NV>
__global__ __launch_bounds__(256) void k_router_fwd(const L *__restrict__ logits, int T, int E, int k, int renorm,
                                                    int32_t *__restrict__ index, float *__restrict__ weight) {
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    float v[NV];
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        v[i] = e < E ? load_logit(logits + (int64_t)t * E + e) : kNegInf;
        key[i] = e < E ? order_key(v[i]) : 0;
    }
    float top = 0.f, mine = kNegInf;   // mine: the logit of slot `lane`
    int pick = -1;
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint64_t c = ((uint64_t)key[i] << 32) | (uint32_t)~(lane + 64 * i);
            best = c > best ? c : best;
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const uint64_t o = __shfl_xor(best, d);
            best = o > best ? o : best;
        }
        const uint32_t bk = (uint32_t)(best >> 32);
        if (bk <= kKeyNegInf) break;   // nothing but -infinity is left
        const int e = (int)~(uint32_t)best;
        float val = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (e == lane + 64 * i) {
                val = v[i];
                key[i] = 0;
            }
        }
        val = __shfl(val, e & 63);
        if (j == 0) top = val;
        if (lane == j) {
            pick = e;
            mine = val;
        }
    }
    // Weights in 32 bits. top is a real logit, +infinity or NaN whenever any slot was filled.
    float ex = pick >= 0 ? expf(mine - top) : 0.f, den = ex;
    if (!renorm) {
        den = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) den += expf(v[i] - top);   // -infinity gives 0
    }
    den = wave_sum(den);
    if (lane < k) {
        index[(int64_t)t * k + lane] = pick;
        weight[(int64_t)t * k + lane] = pick >= 0 ? ex / den : 0.f;
    }
}

// Router backward, one wave a token. Not renormalised: p is computed again from the logits.
template <typename L, int NV>
__global__ __launch_bounds__(256) void k_router_bwd(const L *__restrict__ logits, int T, int E, int k, int renorm,
                                                    const int32_t *__restrict__ index, const float *__restrict__ weight,
                                                    const float *__restrict__ dweight, L *__restrict__ dlogits) {
    const int lane = threadIdx.x & 63, t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    int pick = -1;
    float w = 0.f, g = 0.f;
    if (lane < k) {
        pick = index[(int64_t)t * k + lane];
        if ((unsigned)pick < (unsigned)E) {
            w = weight[(int64_t)t * k + lane];
            g = dweight[(int64_t)t * k + lane];
        } else {
            pick = -1;
        }
    }
    const float inner = wave_sum(w * g);
    float v[NV], d[NV];
    if (!renorm) {
        float m = kNegInf;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 64 * i;
            v[i] = e < E ? load_logit(logits + (int64_t)t * E + e) : kNegInf;
            nan |= v[i] != v[i];
            m = fmaxf(m, v[i]);
        }
#pragma unroll
        for (int o = 32; o; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
        if (__any(nan)) m = __builtin_nanf("");
        const bool none = m == kNegInf;
        float den = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            v[i] = none ? 0.f : expf(v[i] - m);
            den += v[i];
        }
        den = wave_sum(den);
        const float scale = none ? 0.f : 1.f / den;
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = -(v[i] * scale) * inner;
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = 0.f;
    }
    const float add = renorm ? w * (g - inner) : w * g;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl(pick, j);
        const float a = __shfl(add, j);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (e == lane + 64 * i) d[i] += a;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        if (e < E) store_logit(dlogits + (int64_t)t * E + e, d[i]);
    }
}

// ------------------------------------------------------------------------------------------
// The plan: a stable counting sort of S = T k slots by expert.
// Chunks of 1024 slots (16 waves): a slot's row is offsets[e] + the slots of e in earlier chunks + those in
// earlier waves of the chunk + those in lower lanes of its wave (a ballot for each bit of e).
// Up to one chunk, one work-group does everything; beyond that, a launch counts each chunk, a second one
// turns the counts into first rows and offsets, and a third one writes.
// ------------------------------------------------------------------------------------------
constexpr int kPlanChunk = 1024;

// Counts of this chunk's waves in cnt[16][E] (16-bit) and this slot's rank among its wave's.
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

__global__ __launch_bounds__(kPlanChunk) void k_plan_one(const int32_t *__restrict__ index, int S, int k, int E, int bits,
                                                         int32_t *__restrict__ offsets, int32_t *__restrict__ row_token,
                                                         int32_t *__restrict__ slot_row) {
    extern __shared__ uint16_t cnt[];   // [16][E]
    __shared__ int scratch[16];
    __shared__ int first[kMaxExperts];
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < 16 * E; i += kPlanChunk) cnt[i] = 0;
    __syncthreads();
    const int e = plan_expert(index, tid, S, E);
    const int rank = plan_rank(e, E, bits, cnt);
    __syncthreads();
    int mine = 0;
    if (tid < E) {
        for (int w = 0; w < 16; ++w) {
            const int c = cnt[w * E + tid];
            cnt[w * E + tid] = (uint16_t)mine;
            mine += c;
        }
    }
    int live;
    const int before = block_prefix(mine, scratch, &live);
    if (tid < E) {
        first[tid] = before;
        offsets[tid] = before;
    }
    if (tid == 0) offsets[E] = live;
    __syncthreads();
    if (tid < S) {
        const int row = e < E ? first[e] + cnt[wave * E + e] + rank : -1;
        slot_row[tid] = row;
        if (row >= 0) row_token[row] = tid / k;
        if (tid >= live) row_token[tid] = -1;
    }
}

__global__ __launch_bounds__(kPlanChunk) void k_plan_count(const int32_t *__restrict__ index, int64_t S, int E,
                                                           int32_t *__restrict__ counts) {
    __shared__ int hist[kMaxExperts];
    const int tid = threadIdx.x;
    for (int i = tid; i < E; i += kPlanChunk) hist[i] = 0;
    __syncthreads();
    const int e = plan_expert(index, (int64_t)blockIdx.x * kPlanChunk + tid, S, E);
    if (e < E) atomicAdd(&hist[e], 1);   // whole numbers: the order does not matter
    __syncthreads();
    for (int i = tid; i < E; i += kPlanChunk) counts[(int64_t)blockIdx.x * E + i] = hist[i];
}

// counts[chunk][e] -> the rows of e in earlier chunks; offsets from the totals. One work-group.
__global__ __launch_bounds__(kPlanChunk) void k_plan_first(int32_t *__restrict__ counts, int chunks, int E,
                                                           int32_t *__restrict__ offsets) {
    __shared__ int scratch[16];
    const int tid = threadIdx.x;
    int mine = 0;
    if (tid < E) {
        for (int c = 0; c < chunks; ++c) {
            const int n = counts[(int64_t)c * E + tid];
            counts[(int64_t)c * E + tid] = mine;
            mine += n;
        }
    }
    int live;
    const int before = block_prefix(mine, scratch, &live);
    if (tid < E) offsets[tid] = before;
    if (tid == 0) offsets[E] = live;
}

__global__ __launch_bounds__(kPlanChunk) void k_plan_write(const int32_t *__restrict__ index, int64_t S, int k, int E,
                                                           int bits, const int32_t *__restrict__ counts,
                                                           const int32_t *__restrict__ offsets,
                                                           int32_t *__restrict__ row_token,
                                                           int32_t *__restrict__ slot_row) {
    extern __shared__ uint16_t cnt[];   // [16][E]
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int i = tid; i < 16 * E; i += kPlanChunk) cnt[i] = 0;
    __syncthreads();
    const int64_t s = (int64_t)blockIdx.x * kPlanChunk + tid;
    const int e = plan_expert(index, s, S, E);
    const int rank = plan_rank(e, E, bits, cnt);
    __syncthreads();
    if (s >= S) return;
    int row = -1;
    if (e < E) {
        row = offsets[e] + counts[(int64_t)blockIdx.x * E + e] + rank;
        for (int w = 0; w < wave; ++w) row += cnt[w * E + e];
    }
    slot_row[s] = row;
    if (row >= 0) row_token[row] = (int32_t)(s / k);
    if (s >= offsets[E]) row_token[s] = -1;
}

// ------------------------------------------------------------------------------------------
// The sum over a token's rows and its gradient: 8 columns a thread.
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

__global__ __launch_bounds__(256) void k_combine_fwd(const uint16_t *__restrict__ Y, int T, int k, int N, int R,
                                                     const int32_t *__restrict__ slot_row,
                                                     const float *__restrict__ weight, uint16_t *__restrict__ out) {
    const int n8 = N >> 3;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)T * n8) return;
    const int t = (int)(i / n8), c = (int)(i % n8);
    float acc[8] = {};
    for (int j = 0; j < k; ++j) {
        const int row = slot_row[(int64_t)t * k + j];
        if ((unsigned)row >= (unsigned)R) continue;
        const float w = weight ? weight[(int64_t)t * k + j] : 1.f;
        float y[8];
        unpack8(*reinterpret_cast<const u32x4 *>(Y + (int64_t)row * N + c * 8), y);
#pragma unroll
        for (int v = 0; v < 8; ++v) acc[v] += w * y[v];
    }
    *reinterpret_cast<u32x4 *>(out + (int64_t)t * N + c * 8) = pack8(acc);
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
    const dim3 grid((unsigned)((T + 3) / 4)), block(256);
    const L *lg = static_cast<const L *>(logits);
    auto run = [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        if (fwd)
            hipLaunchKernelGGL((k_router_fwd<L, NV>), grid, block, 0, st, lg, T, E, k, (int)renorm, index, weight);
        else
            hipLaunchKernelGGL((k_router_bwd<L, NV>), grid, block, 0, st, lg, T, E, k, (int)renorm, index, weight,
                               dweight, static_cast<L *>(dlogits));
    };
    if (E <= 64) run(std::integral_constant<int, 1>{});
    else if (E <= 128) run(std::integral_constant<int, 2>{});
    else if (E <= 256) run(std::integral_constant<int, 4>{});
    else run(std::integral_constant<int, 16>{});
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

size_t expert_plan_workspace_bytes(int64_t slots, int E) {
    if (slots <= kPlanChunk) return 0;
    return (size_t)((slots + kPlanChunk - 1) / kPlanChunk) * E * sizeof(int32_t);
}

int32_t launch_expert_plan(const int32_t *index, int T, int k, int E, int32_t *offsets, int32_t *row_token,
                           int32_t *slot_row, void *workspace, void *stream) {
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t S = (int64_t)T * k;
    const int bits = bits_for(E);
    const size_t lds = 16 * (size_t)E * sizeof(uint16_t);
    if (S <= kPlanChunk) {
        hipLaunchKernelGGL(k_plan_one, dim3(1), dim3(kPlanChunk), lds, st, index, (int)S, k, E, bits, offsets, row_token,
                           slot_row);
        return launched("bsr_expert_plan");
    }
    const int chunks = (int)((S + kPlanChunk - 1) / kPlanChunk);
    int32_t *counts = static_cast<int32_t *>(workspace);
    hipLaunchKernelGGL(k_plan_count, dim3(chunks), dim3(kPlanChunk), 0, st, index, S, E, counts);
    hipLaunchKernelGGL(k_plan_first, dim3(1), dim3(kPlanChunk), 0, st, counts, chunks, E, offsets);
    hipLaunchKernelGGL(k_plan_write, dim3(chunks), dim3(kPlanChunk), lds, st, index, S, k, E, bits, counts, offsets,
                       row_token, slot_row);
    return launched("bsr_expert_plan");
}

int32_t launch_combine_fwd(const uint16_t *Y, int T, int k, int N, const int32_t *slot_row, const float *weight,
                           uint16_t *out, void *stream) {
    const int64_t n = (int64_t)T * (N / 8);
    hipLaunchKernelGGL(k_combine_fwd, dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                       static_cast<hipStream_t>(stream), Y, T, k, N, T * k, slot_row, weight, out);
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
