// b128_gemm.hip -- the block-scaled FP8 product, plain and grouped by expert.
//
//   out[i,n] = act( sum_kb 2^(sx[t,kb]-127) * 2^(sw[n/128,kb]-127)
//                     * sum_{k in kb} xq[t,k] * wq[n,k]  + bias[n] )
//
// with t = i, or row_idx[i].  The scales are the E8M0 bytes that
// v_mfma_scale_f32_*_f8f6f4 takes per 32 elements of K, so the matrix cores
// apply them while they multiply: a block of 128 gives the same byte to its
// four groups of 32, and no instruction outside the MFMA touches a scale.
#include "b128.h"

namespace llmint8 {
namespace {   // internal linkage: nothing here is exported from the library

// Bounds of expert e's rows, kept inside [0, M] whatever the array holds.
__device__ __forceinline__ void group_bounds(const B128Args &a, int e, int &lo, int &hi)
{
    const int M = (int)a.M;
    lo = min(max(a.offsets[e], 0), M);
    hi = min(max(a.offsets[e + 1], lo), M);
}

// The tile_m-th tile of `bm` rows over all experts' rows (each expert's rows
// start a tile of their own): its expert, first row and the end of the
// expert's rows; false past the last tile.  A wavefront counts the tiles of
// 64 experts at a time.
__device__ __forceinline__ bool find_tile(const B128Args &a, int bm, int tile_m, int lane, int &e,
                                          int &m0, int &mend)
{
    if (!a.offsets) {
        e = 0;
        m0 = tile_m * bm;
        mend = (int)a.M;
        return m0 < mend;
    }
    int before = 0;
    for (int base = 0; base < a.E; base += kWave) {
        int lo = 0, hi = 0;
        if (base + lane < a.E)
            group_bounds(a, base + lane, lo, hi);
        int sum = (hi - lo + bm - 1) / bm;
        const int own = sum;
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const int up = __shfl_up(sum, off, kWave);
            sum += lane >= off ? up : 0;
        }
        const unsigned long long hit = __ballot(before + sum > tile_m);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            e = base + l;
            const int first = before + __shfl(sum - own, l, kWave);
            lo = __shfl(lo, l, kWave);
            mend = __shfl(hi, l, kWave);
            m0 = lo + (tile_m - first) * bm;
            return true;
        }
        before += __shfl(sum, kWave - 1, kWave);
    }
    return false;
}

__device__ __forceinline__ float bias_value(const B128Args &a, int64_t i)
{
    return a.type == kTypeBf16 ? t2f<kTypeBf16>(a.bias[i]) : h2f(a.bias[i]);
}
__device__ __forceinline__ uint16_t out_value(const B128Args &a, float v)
{
    v = a.act && v < 0.0f ? 0.0f : v;   // keeps a NaN
    return a.type == kTypeBf16 ? f2t<kTypeBf16>(v) : f2h(v);
}

// 16 rows x 64 columns per block, a wavefront per 16 columns, operands
// straight from memory: v_mfma_scale_f32_16x16x128_f8f6f4, one block of K per
// instruction.  Lane l holds 32 consecutive bytes (group l/16 of the block) of
// row l%16 of each operand; in a last block of 64 the upper two groups are 0.
__global__ __launch_bounds__(256) void k_matmul_b128(B128Args a, int ntn)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int tn = blockIdx.x % ntn, tm = blockIdx.x / ntn;
    int e, m0, mend;
    if (!find_tile(a, 16, tm, lane, e, m0, mend))
        return;
    const int64_t n0 = (int64_t)tn * 64 + wave * 16;
    const int r = lane % 16, g = lane / 16;
    const int64_t pitch = b128_pitch(a.K);
    int64_t t = m0 + r < mend ? m0 + r : mend - 1;
    if (a.row_idx)
        t = min(max((int64_t)a.row_idx[t], (int64_t)0), a.rows - 1);
    const uint8_t *xp = a.Xq + t * a.K + 32 * g;
    const uint8_t *sx = a.SX + t * pitch;
    const uint8_t *wp = a.CB + ((int64_t)e * a.N + n0 + r) * a.K + 32 * g;
    const uint8_t *sw = a.SB + ((int64_t)e * ((a.N + kB128 - 1) / kB128) + n0 / kB128) * pitch;
    v4f acc = {0, 0, 0, 0};
    for (int64_t k = 0; k < a.K; k += kB128) {
        v4i x0 = {0, 0, 0, 0}, x1 = x0, w0 = x0, w1 = x0;
        if (k + 32 * g < a.K) {
            x0 = *reinterpret_cast<const v4i *>(xp + k);
            x1 = *reinterpret_cast<const v4i *>(xp + k + 16);
            w0 = *reinterpret_cast<const v4i *>(wp + k);
            w1 = *reinterpret_cast<const v4i *>(wp + k + 16);
        }
        const v8i x = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        const v8i w = {w0[0], w0[1], w0[2], w0[3], w1[0], w1[1], w1[2], w1[3]};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 0, 0, 0, sw[k / kB128],
                                                               0, sx[k / kB128]);
    }
    // lane l holds row l%16, columns 4*(l/16) .. +3
    if (m0 + r < mend) {
        const int64_t n = n0 + 4 * g;
        uint16_t v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = out_value(a, acc[q] + (a.bias ? bias_value(a, e * a.N + n + q) : 0.0f));
        *reinterpret_cast<uint2 *>(a.out + (int64_t)(m0 + r) * a.N + n) =
            make_uint2(v[0] | (unsigned)v[1] << 16, v[2] | (unsigned)v[3] << 16);
    }
}

}  // namespace

size_t b128_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_matmul_b128(const B128Args &a, void *, hipStream_t s)
{
    const int64_t ntn = a.N / 64;
    const int64_t ntm = a.offsets ? a.M / 16 + a.E : (a.M + 15) / 16;
    hipLaunchKernelGGL(k_matmul_b128, dim3((unsigned)(ntm * ntn)), dim3(256), 0, s, a, (int)ntn);
    return hipGetLastError();
}

}  // namespace llmint8
