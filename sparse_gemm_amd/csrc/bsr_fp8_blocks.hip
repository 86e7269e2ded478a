// bsr_fp8_blocks.hip -- quantisation to 8-bit floating point with a scale for each block of 128 and back
// (include/bsr_fp8_blocks.h). Bound by the bytes: 2 read and 1 written a value, 1 more for transposed codes, 2 more for values.
#include <hip/hip_runtime.h>

#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_fp8_device.hpp"

namespace bsr {
namespace {

using namespace dev;

// 16 bytes; Stream: as data that is not used again (see streams()).
template <bool Stream>
__device__ __forceinline__ u32x4 load16(const void *p) {
    const u32x4 *v = static_cast<const u32x4 *>(p);
    return Stream ? __builtin_nontemporal_load(v) : *v;
}

// 8 elements a thread and row, 16 threads a group, a wave the 512 columns of `Rows` rows whose scale bytes lie side by side.
// Threads past K only write the zero bytes of their groups. 16384 x 4096: 39 us, 5.2 TB/s; with one row a wave 46.
template <int Rows>
__global__ __launch_bounds__(256) void k_fp8_rows_quantize(const uint16_t *__restrict__ X, int64_t rows, int K, int chunks,
                                                           uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                           uint16_t *__restrict__ values) {
    const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), row = i / chunks * Rows;   // chunk, row by row
    if (row >= rows) return;
    const int cb = (int)(i % chunks), part = threadIdx.x & 63, col = cb * 512 + part * 8;
    const bool real = col - (part & 15) * 8 < K;   // a group that exists
    u32x4 x[Rows];
#pragma unroll
    for (int r = 0; r < Rows; ++r) {
        x[r] = u32x4{0, 0, 0, 0};
        if (col < K && row + r < rows) x[r] = *reinterpret_cast<const u32x4 *>(X + (row + r) * K + col);
    }
#pragma unroll
    for (int r = 0; r < Rows; ++r) {
        if (row + r >= rows) return;
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fp8_top(top, x[r][j]);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
        const int byte = real ? fp8_scale_byte(top) : 0;
        if ((part & 15) == 0) scales[((int64_t)cb * rows + row + r) * 4 + (part >> 4)] = (uint8_t)byte;
        if (col < K) {
            const float scale = mx4_scale_bits((uint32_t)byte);
            const uint2 c = make_uint2(fp8_quantize4(x[r][0], x[r][1], scale), fp8_quantize4(x[r][2], x[r][3], scale));
            *reinterpret_cast<uint2 *>(codes + (row + r) * K + col) = c;
            if (values) *reinterpret_cast<bf16x8 *>(values + (row + r) * K + col) = fp8_expand8(c, scale);
        }
    }
}

// One 128 x 128 block a work-group: thread t holds rows 8 (t / 16) + 0 .. 7 of the 8 columns from 8 (t % 16), so that a
// transposed row's 8 codes come from its own registers. 8 x 4096 x 4096 with transposed codes: 98 us, 5.5 TB/s; with W left in the caches
// 112, with codes stored as not used again either 101.
template <bool Stream>
__global__ __launch_bounds__(256) void k_fp8_blocks_quantize(const uint16_t *__restrict__ W, int N, int K, int nb, int kb,
                                                             uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                             uint8_t *__restrict__ codes_t, uint8_t *__restrict__ scales_t) {
    __shared__ uint32_t part[4];
    const int k_blk = blockIdx.x % kb, n_blk = blockIdx.x / kb % nb;
    const int64_t e = blockIdx.x / kb / nb, at = e * N * K;
    const int r0 = n_blk * 128 + (threadIdx.x >> 4) * 8, c0 = k_blk * 128 + (threadIdx.x & 15) * 8;
    const bool in = r0 < N && c0 < K;   // N and K are multiples of 8
    u32x4 x[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = u32x4{0, 0, 0, 0};
        if (in) x[i] = load16<Stream>(W + at + (int64_t)(r0 + i) * K + c0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fp8_top(top, x[i][j]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    const int byte = fp8_scale_byte(top);
    if (threadIdx.x == 0) {
        scales[(e * nb + n_blk) * kb + k_blk] = (uint8_t)byte;
        if (scales_t) scales_t[(e * kb + k_blk) * nb + n_blk] = (uint8_t)byte;
    }
    if (!in) return;
    const float scale = mx4_scale_bits((uint32_t)byte);
    uint32_t c[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i][0] = fp8_quantize4(x[i][0], x[i][1], scale);
        c[i][1] = fp8_quantize4(x[i][2], x[i][3], scale);
        *reinterpret_cast<uint2 *>(codes + at + (int64_t)(r0 + i) * K + c0) = make_uint2(c[i][0], c[i][1]);
    }
    if (!codes_t) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {   // columns c0 + 4 q + 0 .. 3
        const uint32_t lo[4] = {c[0][q], c[1][q], c[2][q], c[3][q]}, hi[4] = {c[4][q], c[5][q], c[6][q], c[7][q]};
        uint32_t tl[4], th[4];
        transpose4(lo, tl);
        transpose4(hi, th);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2 *>(codes_t + at + (int64_t)(c0 + 4 * q + j) * N + r0) = make_uint2(tl[j], th[j]);
    }
}

// 8 codes a thread. rowwise: scales of bsr_fp8_dequantize_rows, else of one expert's blocks after the other. 8 x 4096 x 4096: 70 us,
// 5.8 TB/s; right behind their quantisation, which leaves the codes in the caches, 58, without Stream 71.
template <bool Rowwise, bool Stream>
__global__ __launch_bounds__(256) void k_fp8_dequantize(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                        int64_t rows, int N, int K, uint16_t *__restrict__ values) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / (K / 8);   // K / 8 pieces a row
    if (row >= rows) return;
    const int col = (int)(i % (K / 8)) * 8, g = col >> 7;
    int64_t s;
    if constexpr (Rowwise) {
        s = ((int64_t)(g >> 2) * rows + row) * 4 + (g & 3);
    } else {
        const int64_t e = row / N;
        s = (e * ((N + 127) / 128) + ((int)(row % N) >> 7)) * ((K + 127) / 128) + g;
    }
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 *from = reinterpret_cast<const u32x2 *>(codes + i * 8);
    u32x4 *to = reinterpret_cast<u32x4 *>(values + i * 8);
    const u32x2 c = Stream ? __builtin_nontemporal_load(from) : *from;
    const u32x4 v = __builtin_bit_cast(u32x4, fp8_expand8(make_uint2(c[0], c[1]), mx4_scale_bits(scales[s])));
    if constexpr (Stream) __builtin_nontemporal_store(v, to);
    else *to = v;
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

template <bool Rowwise>
int32_t dequantize(const char *what, const uint8_t *codes, const uint8_t *scales, int64_t rows, int N, int K, uint16_t *values,
                   void *stream) {
    const int64_t blocks = (rows * (K / 8) + 255) / 256;
    if (const int32_t bad = check_grid(blocks, 256, what)) return bad;
    hipLaunchKernelGGL((streams(rows * K * 2, true) ? k_fp8_dequantize<Rowwise, true> : k_fp8_dequantize<Rowwise, false>),
                       dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), codes, scales, rows, N, K, values);
    return launched(what);
}

}  // namespace

int32_t launch_fp8_quantize_rows(const uint16_t *X, int64_t rows, int K, uint8_t *codes, uint8_t *scales, uint16_t *values,
                                 void *stream) {
    const char *what = "bsr_fp8_quantize_rows";
    const int chunks = (K + 511) / 512;
    // four rows a wave where that leaves every CU eight waves
    const int each = rows * chunks >= 32 * kCUs ? 4 : 1;
    const int64_t blocks = ((rows + each - 1) / each * chunks + 3) / 4;
    if (const int32_t bad = check_grid(blocks, 256, what)) return bad;
    hipLaunchKernelGGL((each == 4 ? k_fp8_rows_quantize<4> : k_fp8_rows_quantize<1>), dim3((unsigned)blocks), dim3(256), 0,
                       static_cast<hipStream_t>(stream), X, rows, K, chunks, codes, scales, values);
    return launched(what);
}

int32_t launch_fp8_quantize_blocks(const uint16_t *W, int E, int N, int K, uint8_t *codes, uint8_t *scales, uint8_t *codes_t,
                                   uint8_t *scales_t, void *stream) {
    const char *what = "bsr_fp8_quantize_blocks";
    const int nb = (N + 127) / 128, kb = (K + 127) / 128;
    const int64_t blocks = (int64_t)E * nb * kb;
    if (const int32_t bad = check_grid(blocks, 256, what)) return bad;
    hipLaunchKernelGGL((streams((int64_t)E * N * K * 2, K % 64 == 0) ? k_fp8_blocks_quantize<true> : k_fp8_blocks_quantize<false>),
                       dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), W, N, K, nb, kb, codes, scales, codes_t,
                       scales_t);
    return launched(what);
}

int32_t launch_fp8_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint16_t *values, void *stream) {
    return dequantize<true>("bsr_fp8_dequantize_rows", codes, scales, rows, 1, K, values, stream);
}

int32_t launch_fp8_dequantize_blocks(const uint8_t *codes, const uint8_t *scales, int E, int N, int K, uint16_t *values,
                                     void *stream) {
    return dequantize<false>("bsr_fp8_dequantize_blocks", codes, scales, (int64_t)E * N, N, K, values, stream);
}

}  // namespace bsr
