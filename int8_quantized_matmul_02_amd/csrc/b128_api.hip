// b128_api.hip -- the C ABI of the block-scaled FP8 operators: argument checks
// and dispatch (documented in include/llmint8.h).

#include <math.h>

#include "../../include/llmint8_test.h"
#include "b128.h"

using namespace llmint8;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned8(const void *p) { return ((uintptr_t)p & 7u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
bool bad_type(int t) { return t != LLMINT8_F16 && t != LLMINT8_BF16; }
bool bad_act(int a) { return a != LLMINT8_ACT_NONE && a != LLMINT8_ACT_RELU; }

bool bad_path(int path, int parts)
{
    return path < 0 || path > kB128Paths || parts < 0 || parts > kB128MostParts;
}

// Sizes the kernels index in 32 bits.
constexpr int64_t kMaxRows = 0x7fff0000;
constexpr int64_t kMaxB128K = 133144;
constexpr int64_t kMaxB128N = (int64_t)1 << 24;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxBlocks = ((int64_t)1 << 24) - 1;   // 128 x 128, of one call to quantize: 550 GB
constexpr int64_t kMaxIndexedBytes = 0xffe00000;   // what a buffer resource covers
constexpr int64_t kMaxOutputs = (int64_t)1 << 38;   // of one product: 512 GB, past the card's memory

llmint8_status_t check_b128(int64_t T, int64_t K, int64_t N, int64_t E)
{
    if (T <= 0 || K <= 0 || N <= 0 || E <= 0)
        return LLMINT8_ERR_INVALID_ARG;
    if (K % 64 != 0 || N % 64 != 0 || K > kMaxB128K || N > kMaxB128N || T > kMaxRows ||
        E > kMaxExperts)
        return LLMINT8_ERR_UNSUPPORTED_SHAPE;
    return LLMINT8_OK;
}

llmint8_status_t status(hipError_t e) { return e == hipSuccess ? LLMINT8_OK : LLMINT8_ERR_HIP; }

// [a, a + bytes) and [b, b + bytes) share a part but are not the same range.
bool partly_overlap(const void *a, const void *b, int64_t bytes)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x != y && (x < y ? y - x : x - y) < (uintptr_t)bytes;
}

}  // namespace

extern "C" {

int64_t llmint8_b128_pitch(int64_t K) { return K <= 0 ? 0 : b128_pitch(K); }

llmint8_status_t llmint8_rmsnorm_b128(const uint16_t *X, const uint16_t *residual,
                                      const uint16_t *gamma, int type, int64_t T, int64_t K,
                                      float eps, uint8_t *Xq8, uint8_t *SX,
                                      uint16_t *residual_out, uint16_t *Y, hipStream_t stream)
{
    if (!X || !gamma || !Xq8 || !SX || !aligned16(X) || !aligned16(residual) ||
        !aligned16(gamma) || !aligned16(Xq8) || !aligned4(SX) || !aligned16(residual_out) ||
        !aligned16(Y) || (residual_out && !residual) || bad_type(type) || !isfinite(eps) ||
        eps < 0.0f)
        return LLMINT8_ERR_INVALID_ARG;
    const llmint8_status_t st = check_b128(T, K, 64, 1);
    if (st != LLMINT8_OK)
        return st;
    // in place is fine (a thread reads its elements before it writes them), a
    // shifted overlap is not
    const int64_t bytes = 2 * T * K;
    if (partly_overlap(residual_out, residual, bytes) || partly_overlap(residual_out, X, bytes) ||
        partly_overlap(Y, X, bytes) || partly_overlap(Y, residual, bytes) || (Y && Y == residual_out) ||
        partly_overlap(Y, residual_out, bytes))
        return LLMINT8_ERR_INVALID_ARG;
    return status(launch_rmsnorm_b128(
        RmsNormArgs{X, residual, gamma, residual_out, Y, T, K, eps, Xq8, SX}, type, stream));
}

llmint8_status_t llmint8_quantize_act_b128(const uint16_t *X, int type, int64_t T, int64_t K,
                                           uint8_t *Xq8, uint8_t *SX, hipStream_t stream)
{
    if (!X || !Xq8 || !SX || !aligned16(X) || !aligned16(Xq8) || !aligned4(SX) || bad_type(type))
        return LLMINT8_ERR_INVALID_ARG;
    const llmint8_status_t st = check_b128(T, K, 64, 1);
    if (st != LLMINT8_OK)
        return st;
    return status(launch_quantize_act_b128(X, T, K, type, Xq8, SX, stream));
}

llmint8_status_t llmint8_quantize_weight_b128(const uint16_t *W_t, int type, int64_t E, int64_t K,
                                              int64_t N, uint8_t *CB8, uint8_t *SB,
                                              hipStream_t stream)
{
    if (!W_t || !CB8 || !SB || !aligned16(W_t) || !aligned16(CB8) || !aligned4(SB) ||
        bad_type(type))
        return LLMINT8_ERR_INVALID_ARG;
    const llmint8_status_t st = check_b128(1, K, N, E);
    if (st != LLMINT8_OK)
        return st;
    if (E * ((N + kB128 - 1) / kB128) * ((K + kB128 - 1) / kB128) > kMaxBlocks)
        return LLMINT8_ERR_UNSUPPORTED_SHAPE;
    return status(launch_quantize_weight_b128(W_t, E, N, K, type, CB8, SB, stream));
}

size_t llmint8_matmul_b128_workspace_bytes_path(int64_t T, int64_t K, int64_t N, int path,
                                                int parts)
{
    return check_b128(T, K, N, 1) == LLMINT8_OK && T * N <= kMaxOutputs && !bad_path(path, parts)
               ? b128_workspace_bytes(T, K, N, path, parts)
               : 0;
}

size_t llmint8_matmul_b128_workspace_bytes(int64_t T, int64_t K, int64_t N)
{
    return llmint8_matmul_b128_workspace_bytes_path(T, K, N, 0, 0);
}

llmint8_status_t llmint8_matmul_b128_path(const uint8_t *Xq8, const uint8_t *SX, int64_t T,
                                          int64_t K, int64_t N, const uint8_t *CB8,
                                          const uint8_t *SB, const uint16_t *bias, int activation,
                                          int type, uint16_t *out, void *ws, size_t ws_bytes,
                                          int path, int parts, hipStream_t stream)
{
    if (!Xq8 || !SX || !CB8 || !SB || !out || !aligned16(Xq8) || !aligned4(SX) ||
        !aligned16(CB8) || !aligned4(SB) || !aligned8(bias) || !aligned16(out) ||
        !aligned16(ws) || bad_act(activation) || bad_type(type) || bad_path(path, parts))
        return LLMINT8_ERR_INVALID_ARG;
    const llmint8_status_t st = check_b128(T, K, N, 1);
    if (st != LLMINT8_OK)
        return st;
    if (T * N > kMaxOutputs)
        return LLMINT8_ERR_UNSUPPORTED_SHAPE;
    const size_t need = b128_workspace_bytes(T, K, N, path, parts);
    if (need && (!ws || ws_bytes < need))
        return LLMINT8_ERR_WORKSPACE;
    return status(launch_matmul_b128(
        B128Args{Xq8, SX, CB8, SB, bias, out, T, T, K, N, activation, type}, ws, path, parts,
        stream));
}

llmint8_status_t llmint8_matmul_b128(const uint8_t *Xq8, const uint8_t *SX, int64_t T, int64_t K,
                                     int64_t N, const uint8_t *CB8, const uint8_t *SB,
                                     const uint16_t *bias, int activation, int type,
                                     uint16_t *out, void *ws, size_t ws_bytes, hipStream_t stream)
{
    return llmint8_matmul_b128_path(Xq8, SX, T, K, N, CB8, SB, bias, activation, type, out, ws,
                                    ws_bytes, 0, 0, stream);
}

llmint8_status_t llmint8_matmul_grouped_b128_path(const uint8_t *Xq8, const uint8_t *SX, int64_t T,
                                                  int64_t K, int64_t N, const uint8_t *CB8,
                                                  const uint8_t *SB, int64_t E,
                                                  const int32_t *offsets, const int32_t *row_idx,
                                                  int64_t M, const uint16_t *bias, int activation,
                                                  int type, uint16_t *out, int path,
                                                  hipStream_t stream)
{
    if (!Xq8 || !SX || !CB8 || !SB || !offsets || !out || !aligned16(Xq8) || !aligned4(SX) ||
        !aligned16(CB8) || !aligned4(SB) || !aligned4(offsets) || !aligned4(row_idx) ||
        !aligned8(bias) || !aligned16(out) || bad_act(activation) || bad_type(type) ||
        bad_path(path, 1) || M <= 0 ||
        (!row_idx && M != T))
        return LLMINT8_ERR_INVALID_ARG;
    const llmint8_status_t st = check_b128(T, K, N, E);
    if (st != LLMINT8_OK)
        return st;
    // rows read by index are addressed with 32-bit offsets
    if (M > kMaxRows || M * N > kMaxOutputs || (row_idx && T * K > kMaxIndexedBytes))
        return LLMINT8_ERR_UNSUPPORTED_SHAPE;
    return status(launch_matmul_b128(B128Args{Xq8, SX, CB8, SB, bias, out, T, M, K, N, activation,
                                              type, (int)E, offsets, row_idx},
                                     nullptr, path, 1, stream));
}

llmint8_status_t llmint8_matmul_grouped_b128(const uint8_t *Xq8, const uint8_t *SX, int64_t T,
                                             int64_t K, int64_t N, const uint8_t *CB8,
                                             const uint8_t *SB, int64_t E,
                                             const int32_t *offsets, const int32_t *row_idx,
                                             int64_t M, const uint16_t *bias, int activation,
                                             int type, uint16_t *out, hipStream_t stream)
{
    return llmint8_matmul_grouped_b128_path(Xq8, SX, T, K, N, CB8, SB, E, offsets, row_idx, M,
                                            bias, activation, type, out, 0, stream);
}

}  // extern "C"
