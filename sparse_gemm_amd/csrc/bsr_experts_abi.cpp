// bsr_experts_abi.cpp -- the extern "C" entry points of include/bsr_experts.h, bsr_mx4.h, bsr_fp8_blocks.h and bsr_expert_ffn.h:
// argument checks and dispatch. Nothing is enqueued before every argument has been checked; no C++
// exception escapes.
#include <cstdint>
#include <initializer_list>
#include <new>
#include <string>
#include <utility>

#include "bsr_experts_internal.hpp"

namespace bsr {
namespace {

struct Ptr {
    const void *p;
    const char *name;
    bool optional;
    unsigned align;
};

int32_t check_ptrs(std::initializer_list<Ptr> ptrs) {
    for (const Ptr &q : ptrs) {
        if (!q.p && !q.optional) return fail(BSR_ERR_INVALID_ARG, std::string(q.name) + " is NULL");
        if ((uintptr_t)q.p % q.align)
            return fail(BSR_ERR_MISALIGNED, std::string(q.name) + " is not aligned to " + std::to_string(q.align) + " bytes");
    }
    return BSR_OK;
}

int32_t check_slots(int64_t T, int32_t k, int32_t E) {
    if (E < 1 || E > kMaxExperts) return fail(BSR_ERR_INVALID_ARG, "E must lie in [1, 1024], got " + std::to_string(E));
    if (k < 1 || k > kMaxSlots || k > E) return fail(BSR_ERR_INVALID_ARG, "k must lie in [1, min(32, E)], got " + std::to_string(k));
    if (T < 0 || T > kMaxExpertRows / k) return fail(BSR_ERR_INVALID_ARG, "T * k must lie in [0, 2^24]");
    return BSR_OK;
}

int32_t check_logits(int32_t type, int32_t renormalize) {
    if (type != BSR_LOGITS_F32 && type != BSR_LOGITS_BF16) return fail(BSR_ERR_UNSUPPORTED, "logits must be f32 or bf16");
    if (renormalize != 0 && renormalize != 1) return fail(BSR_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    return BSR_OK;
}

// Sizes of a grouped product; bits: 16, 8 or 4 per activation, wbits per weight. by_tile: activations that are not gathered are
// read behind a descriptor of a tile's rows, so that their size has no limit.
int32_t check_product(int64_t T, int64_t R, int32_t E, int32_t N, int32_t K, bool gathered, int bits, int wbits, bool by_tile) {
    if (E < 1 || E > kMaxExperts) return fail(BSR_ERR_INVALID_ARG, "E must lie in [1, 1024], got " + std::to_string(E));
    if (R < 0 || R > kMaxExpertRows) return fail(BSR_ERR_INVALID_ARG, "R must lie in [0, 2^24]");
    if (gathered && (T < 0 || T > kMaxExpertRows)) return fail(BSR_ERR_INVALID_ARG, "T must lie in [0, 2^24]");
    if (N < 8 || N % 8 || N >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "N must be a positive multiple of 8 below 2^20");
    const int kstep = wbits == 4 ? 32 : wbits == 8 ? 16 : 8;
    if (K < kstep || K % kstep || K >= (1 << 20))
        return fail(BSR_ERR_INVALID_ARG, "K must be a positive multiple of " + std::to_string(kstep) + " below 2^20");
    const uint64_t rows = gathered ? (uint64_t)T : by_tile ? 0 : (uint64_t)R;
    if (rows * K * bits / 8 > kMaxOperandBytes)
        return fail(BSR_ERR_INVALID_ARG, "activations of more than 0xF0000000 bytes");
    if ((uint64_t)N * K * wbits / 8 > kMaxOperandBytes)
        return fail(BSR_ERR_INVALID_ARG, "one expert's weight has more than 0xF0000000 bytes");
    return BSR_OK;
}

}  // namespace
}  // namespace bsr

#define BSR_TRY_BEGIN try {
#define BSR_TRY_END                                                             \
    }                                                                           \
    catch (const std::bad_alloc &) {                                            \
        return fail(BSR_ERR_OUT_OF_MEMORY, "host allocation failed");           \
    }                                                                           \
    catch (...) {                                                               \
        return fail(BSR_ERR_INVALID_ARG, "unexpected internal exception");      \
    }

#define BSR_CHECK(expr)                \
    do {                               \
        int32_t _st = (expr);          \
        if (_st != BSR_OK) return _st; \
    } while (0)

extern "C" {

using namespace bsr;

int32_t bsr_router_fwd(const void *logits, int32_t type, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                       int32_t *index, float *weight, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_slots(T, k, E));
    BSR_CHECK(check_logits(type, renormalize));
    const bool none = T == 0;
    BSR_CHECK(check_ptrs({{logits, "logits", none, 16}, {index, "index", none, 16}, {weight, "weight", none, 16}}));
    if (none) return BSR_OK;
    return launch_router_fwd(logits, type, (int)T, E, k, renormalize, index, weight, stream);
    BSR_TRY_END
}

int32_t bsr_router_bwd(const void *logits, int32_t type, int64_t T, int32_t E, int32_t k, int32_t renormalize,
                       const int32_t *index, const float *weight, const float *dweight, void *dlogits, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_slots(T, k, E));
    BSR_CHECK(check_logits(type, renormalize));
    const bool none = T == 0;
    BSR_CHECK(check_ptrs({{logits, "logits", none, 16}, {index, "index", none, 16}, {weight, "weight", none, 16},
                          {dweight, "dweight", none, 16}, {dlogits, "dlogits", none, 16}}));
    if (none) return BSR_OK;
    return launch_router_bwd(logits, type, (int)T, E, k, renormalize, index, weight, dweight, dlogits, stream);
    BSR_TRY_END
}

size_t bsr_expert_plan_workspace(int64_t T, int32_t k, int32_t E) {
    if (E < 1 || E > kMaxExperts || k < 1 || k > kMaxSlots || T < 0 || T > kMaxExpertRows / k) return 0;
    return expert_plan_workspace_bytes(T * k, E);
}

int32_t bsr_expert_plan(const int32_t *index, int64_t T, int32_t k, int32_t E, int32_t *offsets, int32_t *row_token,
                        int32_t *slot_row, void *workspace, size_t ws_bytes, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_slots(T, k, E));
    const bool none = T == 0;
    const size_t need = expert_plan_workspace_bytes(T * k, E);
    BSR_CHECK(check_ptrs({{index, "index", none, 16}, {offsets, "offsets", false, 16}, {row_token, "row_token", none, 16},
                          {slot_row, "slot_row", none, 16}, {workspace, "workspace", need == 0, 4}}));
    if (ws_bytes < need)
        return fail(BSR_ERR_WORKSPACE_TOO_SMALL,
                    "workspace of " + std::to_string(ws_bytes) + " bytes, need " + std::to_string(need));
    return launch_expert_plan(index, (int)T, k, E, offsets, row_token, slot_row, workspace, stream);
    BSR_TRY_END
}

int32_t bsr_expert_fwd(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                       const int32_t *offsets, const int32_t *row_token, const bsr_bf16 *W, const bsr_bf16 *bias,
                       bsr_bf16 *Y, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 16, 16, true));
    const bool none = R == 0;
    BSR_CHECK(check_ptrs({{X, "X", none || (row_token && T == 0), 16}, {offsets, "offsets", none, 16},
                          {row_token, "row_token", true, 16}, {W, "W", none, 16}, {bias, "bias", true, 16},
                          {Y, "Y", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_fwd({(int)T, (int)R, E, N, K, offsets, row_token}, X, W, bias, Y, stream);
    BSR_TRY_END
}

int32_t bsr_expert_bwd_input(const bsr_bf16 *dY, int64_t R, int32_t E, int32_t N, int32_t K, const int32_t *offsets,
                             const bsr_bf16 *W, bsr_bf16 *dX, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(0, R, E, N, K, false, 16, 16, true));
    const bool none = R == 0;
    BSR_CHECK(check_ptrs({{dY, "dY", none, 16}, {offsets, "offsets", none, 16}, {W, "W", none, 16}, {dX, "dX", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_bwd_input({0, (int)R, E, N, K, offsets, nullptr}, dY, W, dX, stream);
    BSR_TRY_END
}

int32_t bsr_expert_bwd_weight(const bsr_bf16 *dY, const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N,
                              int32_t K, const int32_t *offsets, const int32_t *row_token, bsr_bf16 *dW,
                              bsr_bf16 *dbias, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 16, 16, false));
    if ((uint64_t)R * N * 2 > kMaxOperandBytes) return fail(BSR_ERR_INVALID_ARG, "dY of more than 0xF0000000 bytes");
    const bool none = R == 0;   // the gradients are then 0
    BSR_CHECK(check_ptrs({{dY, "dY", none, 16}, {X, "X", none || (row_token && T == 0), 16}, {offsets, "offsets", false, 16},
                          {row_token, "row_token", true, 16}, {dW, "dW", dbias != nullptr, 16}, {dbias, "dbias", true, 16}}));
    return launch_expert_bwd_weight({(int)T, (int)R, E, N, K, offsets, row_token}, dY, X, dW, dbias, stream);
    BSR_TRY_END
}

static int32_t check_combine(int64_t T, int32_t k, int32_t N) {
    BSR_CHECK(check_slots(T, k, kMaxExperts));
    if (N < 8 || N % 8 || N >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "N must be a positive multiple of 8 below 2^20");
    return BSR_OK;
}

int32_t bsr_expert_combine_fwd(const bsr_bf16 *Y, int64_t T, int32_t k, int32_t N, const int32_t *slot_row,
                               const float *weight, bsr_bf16 *out, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_combine(T, k, N));
    const bool none = T == 0;
    BSR_CHECK(check_ptrs({{Y, "Y", none, 16}, {slot_row, "slot_row", none, 16}, {weight, "weight", true, 16},
                          {out, "out", none, 16}}));
    if (none) return BSR_OK;
    return launch_combine_fwd(Y, (int)T, k, N, slot_row, weight, out, stream);
    BSR_TRY_END
}

int32_t bsr_expert_combine_bwd(const bsr_bf16 *dout, const bsr_bf16 *Y, int64_t T, int32_t k, int32_t E, int32_t N,
                               const int32_t *offsets, const int32_t *slot_row, const float *weight, bsr_bf16 *dY,
                               float *dweight, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_slots(T, k, E));
    BSR_CHECK(check_combine(T, k, N));
    const bool none = T == 0;
    BSR_CHECK(check_ptrs({{dout, "dout", none, 16}, {Y, "Y", none, 16}, {offsets, "offsets", none, 16},
                          {slot_row, "slot_row", none, 16}, {weight, "weight", true, 16}, {dY, "dY", none, 16},
                          {dweight, "dweight", none, 16}}));
    if (none) return BSR_OK;
    return launch_combine_bwd(dout, Y, (int)T, k, E, N, offsets, slot_row, weight, dY, dweight, stream);
    BSR_TRY_END
}

static int32_t check_mx4(int64_t rows, int32_t K) {
    if (K < 32 || K % 32 || K >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "K must be a positive multiple of 32 below 2^20");
    if (rows < 0 || rows > INT64_C(0xFFFFFFFFFFF) / K) return fail(BSR_ERR_INVALID_ARG, "rows out of range");
    return BSR_OK;
}

int32_t bsr_mx4_quantize(const bsr_bf16 *X, int64_t rows, int32_t K, uint8_t *codes, uint8_t *scales,
                         bsr_bf16 *values, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_mx4(rows, K));
    const bool none = rows == 0;
    BSR_CHECK(check_ptrs({{X, "X", none, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 16},
                          {values, "values", true, 16}}));
    if (none) return BSR_OK;
    return launch_mx4_quantize(X, rows, K, codes, scales, values, stream);
    BSR_TRY_END
}

int32_t bsr_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t K, bsr_bf16 *values,
                           void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_mx4(rows, K));
    const bool none = rows == 0;
    BSR_CHECK(check_ptrs({{codes, "codes", none, 16}, {scales, "scales", none, 16}, {values, "values", none, 16}}));
    if (none) return BSR_OK;
    return launch_mx4_dequantize(codes, scales, rows, K, values, stream);
    BSR_TRY_END
}

int32_t bsr_expert_fwd_mx4(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                           const int32_t *offsets, const int32_t *row_token, const uint8_t *codes,
                           const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 16, 4, false));
    const bool none = R == 0;
    BSR_CHECK(check_ptrs({{X, "X", none || (row_token && T == 0), 16}, {offsets, "offsets", none, 16},
                          {row_token, "row_token", true, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 16},
                          {bias, "bias", true, 16}, {Y, "Y", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_fwd_mx4({(int)T, (int)R, E, N, K, offsets, row_token}, X, codes, scales, bias, Y, stream);
    BSR_TRY_END
}

int32_t bsr_expert_fwd_mx4_mx4(const uint8_t *xcodes, const uint8_t *xscales, int64_t T, int64_t R, int32_t E,
                               int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_token,
                               const uint8_t *codes, const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y,
                               void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 4, 4, false));
    const bool none = R == 0, nox = none || (row_token && T == 0);
    BSR_CHECK(check_ptrs({{xcodes, "xcodes", nox, 16}, {xscales, "xscales", nox, 16}, {offsets, "offsets", none, 16},
                          {row_token, "row_token", true, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 16},
                          {bias, "bias", true, 16}, {Y, "Y", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_fwd_mx4_mx4({(int)T, (int)R, E, N, K, offsets, row_token}, xcodes, xscales, codes, scales, bias, Y,
                                     stream);
    BSR_TRY_END
}

static int32_t check_fp8_rows(int64_t rows, int32_t K) {
    if (K < 16 || K % 16 || K >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "K must be a positive multiple of 16 below 2^20");
    if (rows < 0 || rows > INT64_C(0xFFFFFFFFFFF) / K) return fail(BSR_ERR_INVALID_ARG, "rows out of range");
    return BSR_OK;
}

int32_t bsr_fp8_quantize_rows(const bsr_bf16 *X, int64_t rows, int32_t K, uint8_t *codes, uint8_t *scales,
                              bsr_bf16 *values, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_fp8_rows(rows, K));
    const bool none = rows == 0;
    BSR_CHECK(check_ptrs({{X, "X", none, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 16},
                          {values, "values", true, 16}}));
    if (none) return BSR_OK;
    return launch_fp8_quantize_rows(X, rows, K, codes, scales, values, stream);
    BSR_TRY_END
}

static int32_t check_fp8_blocks(int32_t E, int32_t N, int32_t K, bool transposed) {
    if (E < 1 || E > kMaxExperts) return fail(BSR_ERR_INVALID_ARG, "E must lie in [1, 1024], got " + std::to_string(E));
    if (K < 16 || K % 16 || K >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "K must be a positive multiple of 16 below 2^20");
    const int step = transposed ? 16 : 8;
    if (N < step || N % step || N >= (1 << 20))
        return fail(BSR_ERR_INVALID_ARG, "N must be a positive multiple of " + std::to_string(step) + " below 2^20");
    return BSR_OK;
}

int32_t bsr_fp8_quantize_blocks(const bsr_bf16 *W, int32_t E, int32_t N, int32_t K, uint8_t *codes, uint8_t *scales,
                                uint8_t *codes_t, uint8_t *scales_t, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_fp8_blocks(E, N, K, codes_t || scales_t));
    const bool plain = !codes_t && !scales_t;
    BSR_CHECK(check_ptrs({{W, "W", false, 16}, {codes, "codes", false, 16}, {scales, "scales", false, 16},
                          {codes_t, "codes_t", plain, 16}, {scales_t, "scales_t", plain, 16}}));
    return launch_fp8_quantize_blocks(W, E, N, K, codes, scales, codes_t, scales_t, stream);
    BSR_TRY_END
}

int32_t bsr_fp8_dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t K, bsr_bf16 *values,
                                void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_fp8_rows(rows, K));
    const bool none = rows == 0;
    BSR_CHECK(check_ptrs({{codes, "codes", none, 16}, {scales, "scales", none, 16}, {values, "values", none, 16}}));
    if (none) return BSR_OK;
    return launch_fp8_dequantize_rows(codes, scales, rows, K, values, stream);
    BSR_TRY_END
}

int32_t bsr_fp8_dequantize_blocks(const uint8_t *codes, const uint8_t *scales, int32_t E, int32_t N, int32_t K,
                                  bsr_bf16 *values, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_fp8_blocks(E, N, K, false));
    BSR_CHECK(check_ptrs({{codes, "codes", false, 16}, {scales, "scales", false, 1}, {values, "values", false, 16}}));
    return launch_fp8_dequantize_blocks(codes, scales, E, N, K, values, stream);
    BSR_TRY_END
}

int32_t bsr_expert_fwd_fp8(const bsr_bf16 *X, int64_t T, int64_t R, int32_t E, int32_t N, int32_t K,
                           const int32_t *offsets, const int32_t *row_token, const uint8_t *codes,
                           const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 16, 8, false));
    const bool none = R == 0;
    BSR_CHECK(check_ptrs({{X, "X", none || (row_token && T == 0), 16}, {offsets, "offsets", none, 16},
                          {row_token, "row_token", true, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 1},
                          {bias, "bias", true, 16}, {Y, "Y", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_fwd_fp8({(int)T, (int)R, E, N, K, offsets, row_token}, X, codes, scales, bias, Y, stream);
    BSR_TRY_END
}

int32_t bsr_expert_fwd_fp8_fp8(const uint8_t *xcodes, const uint8_t *xscales, int64_t T, int64_t R, int32_t E,
                               int32_t N, int32_t K, const int32_t *offsets, const int32_t *row_token,
                               const uint8_t *codes, const uint8_t *scales, const bsr_bf16 *bias, bsr_bf16 *Y,
                               void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_product(T, R, E, N, K, row_token != nullptr, 8, 8, false));
    const bool none = R == 0, nox = none || (row_token && T == 0);
    BSR_CHECK(check_ptrs({{xcodes, "xcodes", nox, 16}, {xscales, "xscales", nox, 16}, {offsets, "offsets", none, 16},
                          {row_token, "row_token", true, 16}, {codes, "codes", none, 16}, {scales, "scales", none, 1},
                          {bias, "bias", true, 16}, {Y, "Y", none, 16}}));
    if (none) return BSR_OK;
    return launch_expert_fwd_fp8_fp8({(int)T, (int)R, E, N, K, offsets, row_token}, xcodes, xscales, codes, scales, bias, Y,
                                     stream);
    BSR_TRY_END
}

static int32_t check_ffn(int32_t T, int32_t dim, int32_t hidden, int32_t E, int32_t k) {
    BSR_CHECK(check_slots(T, k, E));
    if (T > BSR_EXPERT_FFN_TOKENS) return fail(BSR_ERR_INVALID_ARG, "T must be at most " + std::to_string(BSR_EXPERT_FFN_TOKENS));
    if (dim < 8 || dim % 8 || dim >= (1 << 20)) return fail(BSR_ERR_INVALID_ARG, "dim must be a positive multiple of 8 below 2^20");
    if (hidden < 8 || hidden % 8 || hidden >= (1 << 19))
        return fail(BSR_ERR_INVALID_ARG, "hidden must be a positive multiple of 8 below 2^19");
    return BSR_OK;
}

size_t bsr_expert_ffn_workspace(int32_t T, int32_t dim, int32_t hidden, int32_t E, int32_t k) {
    try {
        return check_ffn(T, dim, hidden, E, k) == BSR_OK ? expert_ffn_workspace_bytes(T, dim, hidden, E, k) : 0;
    } catch (...) {
        return 0;
    }
}

int32_t bsr_expert_ffn(const bsr_bf16 *x, int32_t T, int32_t dim, int32_t hidden, int32_t E, int32_t k,
                       int32_t renormalize, const bsr_bf16 *router, int32_t form, const void *up, const uint8_t *up_scales,
                       const void *down, const uint8_t *down_scales, const bsr_bf16 *up_bias, const bsr_bf16 *down_bias,
                       bsr_bf16 *out, void *workspace, size_t ws_bytes, void *stream) {
    BSR_TRY_BEGIN
    BSR_CHECK(check_ffn(T, dim, hidden, E, k));
    BSR_CHECK(check_logits(BSR_LOGITS_F32, renormalize));
    if (form != BSR_WEIGHTS_BF16 && form != BSR_WEIGHTS_MX4 && form != BSR_WEIGHTS_FP8)
        return fail(BSR_ERR_UNSUPPORTED, "weights must be bf16, mx4 or fp8");
    const int step = form == BSR_WEIGHTS_BF16 ? 8 : form == BSR_WEIGHTS_FP8 ? 16 : 32, bits = 128 / step;
    if (dim % step || hidden % step)
        return fail(BSR_ERR_INVALID_ARG, "dim and hidden must be multiples of " + std::to_string(step) + " for weights of this form");
    if ((uint64_t)2 * hidden * dim * bits / 8 > kMaxOperandBytes)
        return fail(BSR_ERR_INVALID_ARG, "one expert's weight has more than 0xF0000000 bytes");
    const bool none = T == 0, bare = form == BSR_WEIGHTS_BF16;
    const unsigned at = form == BSR_WEIGHTS_FP8 ? 1 : 16;   // of scales
    const size_t need = expert_ffn_workspace_bytes(T, dim, hidden, E, k);
    BSR_CHECK(check_ptrs({{x, "x", none, 16}, {router, "router", none, 16}, {up, "up", none, 16},
                          {up_scales, "up_scales", none || bare, at}, {down, "down", none, 16},
                          {down_scales, "down_scales", none || bare, at}, {up_bias, "up_bias", true, 16},
                          {down_bias, "down_bias", true, 16}, {out, "out", none, 16}, {workspace, "workspace", need == 0, 16}}));
    if (ws_bytes < need)
        return fail(BSR_ERR_WORKSPACE_TOO_SMALL,
                    "workspace of " + std::to_string(ws_bytes) + " bytes, need " + std::to_string(need));
    if (none) return BSR_OK;
    return launch_expert_ffn(x, T, dim, hidden, E, k, renormalize != 0, router, form, up, up_scales, down, down_scales, up_bias,
                             down_bias, out, workspace, stream);
    BSR_TRY_END
}

}  // extern "C"
