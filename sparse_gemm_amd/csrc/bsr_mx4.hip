// bsr_mx4.hip -- quantisation to the microscaled 4-bit form and back (include/bsr_mx4.h).
//
// Bound by the bytes: 2 read a value, 17/32 written, 2 more for the values that the codes stand for. 57344 x 4096 with
// values: 176 us, 6.0 TB/s (a copy of 2 GiB: 4.9).
#include <hip/hip_runtime.h>

#include <string>

#include "bsr_experts_internal.hpp"
#include "bsr_mx4_device.hpp"

namespace bsr {
namespace {

using namespace dev;

// 8 elements a thread, 4 neighbouring threads a group, 32 threads a 256-column chunk of one row. Threads
// past K only write the zero bytes of their groups.
__global__ __launch_bounds__(256) void k_quantize(const uint16_t *__restrict__ X, int64_t rows, int K, int chunks,
                                                  uint8_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                  uint16_t *__restrict__ values) {
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);   // chunk, row by row
    if (i >= rows * chunks) return;
    const int64_t row = i / chunks;
    const int cb = (int)(i % chunks), part = threadIdx.x & 31, col = cb * 256 + part * 8;
    u32x4 x = {0, 0, 0, 0};
    if (col < K) x = *reinterpret_cast<const u32x4 *>(X + row * K + col);
    uint32_t top = 0;   // largest magnitude's bits
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const int field = (int)(top >> 7);   // exponent field
    const bool bad = field == 255;
    const int byte = bad ? 255 : max(field - 2, 0);
    const float scale = mx4_scale_bits((uint32_t)byte);
    const uint32_t packed = bad ? 0u : mx4_quantize8(x, scale);
    if ((part & 3) == 0) scales[((int64_t)cb * rows + row) * 8 + (part >> 2)] = (uint8_t)byte;
    if (col < K) {
        *reinterpret_cast<uint32_t *>(codes + (row * K + col) / 2) = packed;
        if (values) {
            *reinterpret_cast<bf16x8 *>(values + row * K + col) = mx4_expand8(packed, scale);
        }
    }
}

// One group a thread.
__global__ __launch_bounds__(256) void k_dequantize(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                                                    int64_t rows, int K, uint16_t *__restrict__ values) {
    const int groups = K / 32;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= rows * groups) return;
    const int64_t row = i / groups;
    const int g = (int)(i % groups);
    const u32x4 c = *reinterpret_cast<const u32x4 *>(codes + i * 16);
    const float scale = mx4_scale_bits(scales[((int64_t)(g >> 3) * rows + row) * 8 + (g & 7)]);
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<bf16x8 *>(values + i * 32 + 8 * q) = mx4_expand8(c[q], scale);
}

int32_t launched(const char *what) {
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return fail(BSR_ERR_HIP, std::string(what) + ": " + hipGetErrorString(err));
    return BSR_OK;
}

}  // namespace

int32_t launch_mx4_quantize(const uint16_t *X, int64_t rows, int K, uint8_t *codes, uint8_t *scales, uint16_t *values,
                            void *stream) {
    const int chunks = (K + 255) / 256;
    const int64_t blocks = (rows * chunks + 7) / 8;
    if (const int32_t bad = check_grid(blocks, 256, "bsr_mx4_quantize")) return bad;
    hipLaunchKernelGGL(k_quantize, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), X, rows, K,
                       chunks, codes, scales, values);
    return launched("bsr_mx4_quantize");
}

int32_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint16_t *values,
                              void *stream) {
    const int64_t blocks = (rows * (K / 32) + 255) / 256;
    if (const int32_t bad = check_grid(blocks, 256, "bsr_mx4_dequantize")) return bad;
    hipLaunchKernelGGL(k_dequantize, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), codes, scales,
                       rows, K, values);
    return launched("bsr_mx4_dequantize");
}

}  // namespace bsr
