// b128.h -- block-scaled FP8: shared definitions of the operators whose E4M3
// operands carry one power-of-two scale per block of 128 (include/llmint8.h,
// "Block-scaled FP8").  Not part of the public ABI.
#pragma once

#include "internal.h"

namespace llmint8 {

constexpr int kB128 = 128;

// Bytes of one row of scales: a byte per block of 128 columns, padded so that
// a row starts on a dword and the scales of four blocks are one load.
__host__ __device__ __forceinline__ int64_t b128_pitch(int64_t K)
{
    return ((K + kB128 - 1) / kB128 + 3) / 4 * 4;
}
constexpr unsigned kB128Pad = 127;   // E8M0 of 1.0, in the padding
constexpr unsigned kE8m0Nan = 255;

// 16-bit element types of the block-scaled operators (LLMINT8_F16, _BF16).
enum { kTypeF16 = 0, kTypeBf16 = 1 };

template <int kT>
__device__ __forceinline__ float t2f(uint16_t u)
{
    if constexpr (kT == kTypeBf16)
        return __builtin_bit_cast(float, (unsigned)u << 16);
    else
        return h2f(u);
}
// To nearest, ties to even.
template <int kT>
__device__ __forceinline__ uint16_t f2t(float f)
{
    if constexpr (kT == kTypeBf16)
        return __builtin_bit_cast(uint16_t, (__bf16)f);
    else
        return f2h(f);
}

// Two values side by side (one conversion instruction where there is one).
template <int kT>
__device__ __forceinline__ unsigned pack2(float a, float b)
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    if constexpr (kT == kTypeBf16)
        return __builtin_bit_cast(unsigned, __builtin_convertvector((f2{a, b}), b2));
    else
        return __builtin_bit_cast(unsigned, __builtin_convertvector((f2{a, b}), h2));
}

// The scale of a block whose largest magnitude has the fp32 bits `a` (sign
// clear): e is the largest integer with a * 2^e <= 448 = 1.75 * 2^8, at most
// 126 so that the stored 2^-e stays a normal fp32; 0 for a = 0.  With
// a = f * 2^E, f in [1, 2): e = 8 - E, one less for f > 1.75.  An infinity or
// NaN makes the whole block NaN: scale byte 255, and every code the NaN that
// x * NaN converts to.
struct B128Scale {
    float mul;       // 2^e
    unsigned byte;   // E8M0 of 2^-e
};
__device__ __forceinline__ B128Scale b128_scale(unsigned a)
{
    if (a >= 0x7f800000u)
        return {__builtin_nanf(""), kE8m0Nan};
    int e = 8 + 127 - (int)(a >> 23) - ((a & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = e < 126 ? e : 126;   // subnormals (exponent field 0) end here too
    e = a == 0 ? 0 : e;
    return {__builtin_bit_cast(float, (unsigned)(e + 127) << 23), (unsigned)(127 - e)};
}

// Eight fp32 values to E4M3 (v_cvt_pk_fp8_f32: nearest, ties to even; scaled
// values are at most 448, so nothing saturates).
__device__ __forceinline__ uint2 cvt8_e4m3(const float (&v)[8])
{
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    return make_uint2((unsigned)lo, (unsigned)hi);
}

// ---- launchers (each enqueues on `s`; return hipGetLastError()) ----
struct RmsNormArgs {
    const uint16_t *X, *R, *G;   // R null: no residual
    uint16_t *H, *Y;             // null: not written
    int64_t T, K;
    float eps;
    uint8_t *Xq, *SX;
};
hipError_t launch_rmsnorm_b128(const RmsNormArgs &a, int type, hipStream_t s);
hipError_t launch_quantize_act_b128(const uint16_t *X, int64_t T, int64_t K, int type,
                                    uint8_t *Xq, uint8_t *SX, hipStream_t s);
hipError_t launch_quantize_weight_b128(const uint16_t *W, int64_t E, int64_t N, int64_t K,
                                       int type, uint8_t *CB, uint8_t *SB, hipStream_t s);

// One product, or (offsets non-null) the products of E experts: output row i
// in [offsets[e], offsets[e+1]) is activation row row_idx[i] (i without
// row_idx) times expert e's weight.
struct B128Args {
    const uint8_t *Xq, *SX;   // [rows, K], [rows, pitch]
    const uint8_t *CB, *SB;   // [E, N, K], [E, ceil(N/128), pitch]
    const uint16_t *bias;     // [E, N] or null
    uint16_t *out;            // [M, N]
    int64_t rows, M, K, N;    // rows of Xq; rows of out (= rows without row_idx)
    int act, type;            // output activation and element type
    int E = 1;
    const int32_t *offsets = nullptr;
    const int32_t *row_idx = nullptr;
    // A plain product may split K: part p takes `per` blocks of K from p * per
    // on and writes fp32 sums to parts [parts, M, N] instead of out.
    int nparts = 1, per = 0;
    float *parts = nullptr;
};
// path: 0, or one of the kernel shapes 1 .. kB128Paths; parts: 0, or into how
// many parts K is split (1 for a grouped product); both 0: the estimate's choice.
constexpr int kB128Paths = 10, kB128MostParts = 8;
hipError_t launch_matmul_b128(const B128Args &a, void *ws, int path, int parts, hipStream_t s);
size_t b128_workspace_bytes(int64_t T, int64_t K, int64_t N, int path, int parts);

}  // namespace llmint8
