// b128_gemm.h -- kernels of the block-scaled FP8 product, plain and grouped by
// expert.
//
//   out[i,n] = act( sum_kb 2^(sx[t,kb]-127) * 2^(sw[n/128,kb]-127)
//                     * sum_{k in kb} xq[t,k] * wq[n,k]  + bias[n] )
//
// with t = i, or row_idx[i].  The scales are the E8M0 bytes that
// v_mfma_scale_f32_*_f8f6f4 takes per 32 elements of K, so the matrix cores
// apply them while they multiply: a block of 128 gives the same byte to its
// four groups of 32, and no instruction outside the MFMA touches a scale but
// to move it.
//
// A launch covers tiles of BM output rows by BN columns.  Rows of one expert
// share its tiles and every expert starts a tile of its own; a plain product
// is the case of one group.  A block finds its tile from the offsets itself
// (a wavefront counts 64 experts' tiles at a time), so the group sizes never
// leave the device; the grid has room for the worst split and blocks past the
// last tile end at once.
//
// Two kernels:
//  * k_b128_big streams 128-byte stages of both operands through an LDS ring
//    into v_mfma_scale_f32_32x32x64 (many rows: bound by the matrix cores);
//  * k_b128_small streams 512-byte stages into v_mfma_scale_f32_16x16x128 and
//    splits each stage's blocks of K over the wavefronts of a block (few rows:
//    bound by reading the weight).
#pragma once

#include "b128.h"
#include "gemm_kernel.h"

namespace llmint8 {
namespace b128 {
namespace {   // internal linkage: nothing here is exported from the library

using gemm::lds_void;
using gemm::wait_vm;

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct Tile {
    int e;            // expert
    int m0, mend;     // first output row, end of the expert's rows
    int64_t n0;
};

// Rows of 64 experts from `base` on: each lane's bounds, kept inside [0, M]
// whatever the array holds, and its number of tiles.
__device__ __forceinline__ int group_tiles(const B128Args &a, int base, int lane, int bm, int &lo,
                                           int &hi)
{
    const int M = (int)a.M;
    lo = hi = 0;
    if (base + lane < a.E) {
        lo = min(max(a.offsets[base + lane], 0), M);
        hi = min(max(a.offsets[base + lane + 1], lo), M);
    }
    return (hi - lo + bm - 1) / bm;
}

__device__ __forceinline__ int wave_prefix_sum(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const int up = __shfl_up(v, off, kWave);
        v += lane >= off ? up : 0;
    }
    return v;
}

// The tile of block `bid`; false for a block past the last one.  Every
// wavefront of the block computes it, from the same data.
template <int BM, int BN, int GROUP>
__device__ __forceinline__ bool find_tile(const B128Args &a, int lane, Tile &t)
{
    const int ntn = (int)((a.N + BN - 1) / BN);
    int tm, tn;
    if (!a.offsets) {
        const int ntm = (int)((a.M + BM - 1) / BM);
        gemm::tile_coords(blockIdx.x, ntm * ntn, ntm, ntn, GROUP, tm, tn);
        t.e = 0;
        t.m0 = tm * BM;
        t.mend = (int)a.M;
        t.n0 = (int64_t)tn * BN;
        return true;
    }
    int ntm = 0, lo, hi;
    for (int base = 0; base < a.E; base += kWave) {
        int n = group_tiles(a, base, lane, BM, lo, hi);
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1)
            n += __shfl_xor(n, off, kWave);
        ntm += n;
    }
    ntm = __builtin_amdgcn_readfirstlane(ntm);
    if ((int)blockIdx.x >= ntm * ntn)
        return false;
    gemm::tile_coords(blockIdx.x, ntm * ntn, ntm, ntn, GROUP, tm, tn);
    t.n0 = (int64_t)tn * BN;
    int before = 0;
    for (int base = 0; base < a.E; base += kWave) {
        const int own = group_tiles(a, base, lane, BM, lo, hi);
        const int sum = wave_prefix_sum(own, lane);
        const unsigned long long hit = __ballot(before + sum > tm);
        if (hit) {
            const int l = __builtin_amdgcn_readfirstlane(__builtin_ctzll(hit));
            const int first = before + __builtin_amdgcn_readlane(sum - own, l);
            t.e = base + l;
            t.m0 = __builtin_amdgcn_readlane(lo, l) + (tm - first) * BM;
            t.mend = __builtin_amdgcn_readlane(hi, l);
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, kWave - 1);
    }
    return false;
}

// The activation row of output row i (rows past the group's end: its last).
__device__ __forceinline__ int64_t source_row(const B128Args &a, const Tile &t, int64_t i)
{
    i = i < t.mend ? i : t.mend - 1;
    if (a.row_idx) {
        const int64_t r = a.row_idx[i];
        return r < 0 ? 0 : r < a.rows ? r : a.rows - 1;
    }
    return i;
}

__device__ __forceinline__ int64_t scale_rows(const B128Args &a) { return (a.N + kB128 - 1) / kB128; }

// One operand's loads: NI instructions of 1 KB per wavefront and stage, each
// through a buffer resource based at `base`, with a fixed 32-bit offset per
// lane and the stage's byte of K as the scalar offset.  Past the end of the
// resource a load gives zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t *base, int64_t bytes)
{
    const uint32_t n = bytes > 0xffffffffll ? 0xffffffffu : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), (short)0, (int)n,
                                             0x00020000);
}

// Activation rows are addressed from the tile's first row, or, read by
// index, from row 0 (the whole matrix is then below 4 GB).
__device__ __forceinline__ int64_t x_base_row(const B128Args &a, const Tile &t)
{
    return a.row_idx ? 0 : t.m0;
}

__device__ __forceinline__ void lds_load4(__amdgpu_buffer_rsrc_t r, lds_void *dst, uint32_t voffset,
                                          uint32_t soffset)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, dst, 4, voffset, soffset, 0, 0);
}

__device__ __forceinline__ unsigned buf_load4(__amdgpu_buffer_rsrc_t r, uint32_t voffset,
                                              uint32_t soffset)
{
    return __builtin_amdgcn_raw_buffer_load_b32(r, voffset, soffset, 0);
}

// Four finished outputs of consecutive columns: bias, activation, rounding.
// An activation keeps a NaN.
template <int kT>
__device__ __forceinline__ uint2 finish4(v4f v, bool bias, uint2 b, int act)
{
    if (bias) {
        v[0] += t2f<kT>((uint16_t)b.x);
        v[1] += t2f<kT>((uint16_t)(b.x >> 16));
        v[2] += t2f<kT>((uint16_t)b.y);
        v[3] += t2f<kT>((uint16_t)(b.y >> 16));
    }
    if (act) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            v[q] = v[q] < 0.0f ? 0.0f : v[q];
    }
    return make_uint2(f2t<kT>(v[0]) | (unsigned)f2t<kT>(v[1]) << 16,
                      f2t<kT>(v[2]) | (unsigned)f2t<kT>(v[3]) << 16);
}

// ---------------------------------------------------------------------------
// Few rows.  BM x BN outputs per block; a stage holds 512 bytes (four blocks
// of K) of each of its BM + BN rows and, with them, the dword of their four
// scales.  Wavefront (wk, wm, wn) multiplies blocks [4/WK * wk, ...) of every
// stage for its FM x FN tiles of 16 x 16; the WK partial sums meet in LDS at
// the end.  One load instruction fetches 512 contiguous bytes of each of two
// rows, which is what HBM wants, and the ring keeps STAGES - 1 stages in
// flight.  The 16-byte chunk c of staged row r sits in slot c ^ (r & 15), so
// that the 16 rows of a fragment read cover all banks.
//
// A lane's 32 bytes of a block are its chunks g and g + 4 (g = lane / 16), the
// same for both operands; in a last block of 64 columns chunks 4 .. 7 are
// replaced by zeros.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_, int WK_, int STAGES_>
struct SmallCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WK = WK_, STAGES = STAGES_;
    static constexpr int GROUP = 4;
    static constexpr int kWaves = WM * WN * WK, kThreads = 64 * kWaves;
    static constexpr int kRowB = 512;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;
    static constexpr int kBlocks = 4 / WK;               // blocks of K per wavefront and stage
    static constexpr int kInstr = (BM + BN) / 2 / kWaves;   // 1 KB loads per wavefront and stage
    static constexpr int kLoads = kInstr + 1;            // and one of scales
    static constexpr int kScaleBytes = kWaves * 256;
    static constexpr int kStageBytes = (BM + BN) * kRowB + kScaleBytes;
    static constexpr int kRing = STAGES * kStageBytes;
    static constexpr int kSumPitch = BN + 4;             // floats per row of the partial sums
    static constexpr int kSums = WK * BM * kSumPitch * 4;
    static constexpr int kLdsBytes = kRing > kSums ? kRing : kSums;
    static_assert(FM >= 1 && FN >= 1 && kBlocks >= 1, "wavefront tile");
    static_assert((BM + BN) / 2 % kWaves == 0, "load split");
    static_assert(BM % 2 == 0 && BM + 1 <= kWaves * 64 && BN <= kB128 && kB128 % BN == 0,
                  "one weight scale row per tile");
    static_assert(STAGES >= 2 && (STAGES - 1) * kLoads < 64, "vmcnt range");
    static_assert(kLdsBytes <= 160 * 1024, "LDS");
};

template <class C>
__global__ __launch_bounds__(C::kThreads) void k_b128_small(B128Args a)
{
    __shared__ __attribute__((aligned(1024))) char smem[C::kLdsBytes];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    Tile t;
    if (!find_tile<C::BM, C::BN, C::GROUP>(a, lane, t))
        return;
    const int wn = wave % C::WN, wm = wave / C::WN % C::WM, wk = wave / (C::WN * C::WM);
    const int64_t pitch = b128_pitch(a.K);
    const int nblk = (int)((a.K + kB128 - 1) / kB128), nst = (nblk + 3) / 4;

    // loads: instruction j of the block's fills staged rows 2j and 2j + 1 (the
    // activations' first)
    const int64_t xr = x_base_row(a, t), wr = (int64_t)t.e * a.N + t.n0;
    const __amdgpu_buffer_rsrc_t rx = resource(a.Xq + xr * a.K, (a.rows - xr) * a.K);
    const __amdgpu_buffer_rsrc_t rw =
        resource(a.CB + wr * a.K, ((int64_t)a.E * a.N - wr) * a.K);
    uint32_t off[C::kInstr];
#pragma unroll
    for (int u = 0; u < C::kInstr; ++u) {
        const int r = 2 * (wave * C::kInstr + u) + lane / 32;
        const int64_t row = r < C::BM ? source_row(a, t, t.m0 + r) - xr : r - C::BM;
        off[u] = (uint32_t)(row * a.K + (((lane % 32) ^ (r & 15)) << 4));
    }
    // scales: slot s of the block's is row s's dword (s < BM), else the weight's
    const __amdgpu_buffer_rsrc_t rsx = resource(a.SX + xr * pitch, (a.rows - xr) * pitch);
    const __amdgpu_buffer_rsrc_t rsw = resource(
        a.SB + ((int64_t)t.e * scale_rows(a) + t.n0 / kB128) * pitch, pitch);
    const int slot = wave * 64 + lane;
    const bool xs = wave * 64 < C::BM;   // this wavefront fetches row scales
    static_assert(C::BM <= 64 || C::BM % 64 == 0, "row scales fill whole wavefronts");
    const uint32_t soff =
        xs ? (uint32_t)((source_row(a, t, t.m0 + (slot < C::BM ? slot : 0)) - xr) * pitch) : 0;

    auto issue = [&](int s) {
        char *st = smem + s % C::STAGES * C::kStageBytes;
        const int sc = s < nst ? s : nst - 1;   // past the end: the last stage again, never read
#pragma unroll
        for (int u = 0; u < C::kInstr; ++u) {
            const int j = wave * C::kInstr + u;
            gemm::lds_load16(2 * j < C::BM ? rx : rw, (lds_void *)(st + j * 1024), off[u],
                             (uint32_t)sc * C::kRowB);
        }
        lds_load4(xs ? rsx : rsw, (lds_void *)(st + (C::BM + C::BN) * C::kRowB + wave * 256), soff,
                  (uint32_t)sc * 4);
    };

    v4f acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            acc[i][j] = v4f{0, 0, 0, 0};

    const int r = lane % 16, g = lane / 16;
    auto frag = [&](const char *row, int blk, bool half) {
        const v4i lo = *reinterpret_cast<const v4i *>(row + (((8 * blk + g) ^ r) << 4));
        v4i hi = *reinterpret_cast<const v4i *>(row + (((8 * blk + g + 4) ^ r) << 4));
        if (half)
            hi = v4i{0, 0, 0, 0};
        return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };

#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s)
        issue(s);
    for (int kt = 0; kt < nst; ++kt) {
        // stage kt has landed for this wavefront, then for all; they are also
        // done reading stage kt - 1, whose buffer stage kt + STAGES - 1 takes
        wait_vm<(C::STAGES - 2) * C::kLoads>();
        __builtin_amdgcn_s_barrier();
        issue(kt + C::STAGES - 1);
        const char *st = smem + kt % C::STAGES * C::kStageBytes;
        const char *sa = st + (wm * C::FM * 16 + r) * C::kRowB;
        const char *sb = st + (C::BM + wn * C::FN * 16 + r) * C::kRowB;
        const unsigned *sc = reinterpret_cast<const unsigned *>(st + (C::BM + C::BN) * C::kRowB);
        unsigned sx[C::FM];
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            sx[i] = sc[wm * C::FM * 16 + i * 16 + r] >> (8 * C::kBlocks * wk);
        const unsigned sw = sc[C::BM <= 64 ? 64 : C::BM] >> (8 * C::kBlocks * wk);
#pragma unroll
        for (int b = 0; b < C::kBlocks; ++b) {
            const int blk = C::kBlocks * wk + b;
            if (4 * kt + blk < nblk) {
                const bool half = (int64_t)(4 * kt + blk) * kB128 + 64 == a.K;
                v8i fa[C::FM], fb[C::FN];
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
                    fa[i] = frag(sa + i * 16 * C::kRowB, blk, half);
#pragma unroll
                for (int j = 0; j < C::FN; ++j)
                    fb[j] = frag(sb + j * 16 * C::kRowB, blk, half);
#pragma unroll
                for (int i = 0; i < C::FM; ++i)
#pragma unroll
                    for (int j = 0; j < C::FN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            fb[j], fa[i], acc[i][j], 0, 0, 0, sw >> (8 * b), 0, sx[i] >> (8 * b));
            }
        }
    }
    wait_vm<0>();                    // the tail loads have landed
    __syncthreads();                 // and nobody reads the ring any more

    // partial sums: lane holds row r, columns 4g .. 4g + 3 of each tile
    float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
            *reinterpret_cast<v4f *>(sums +
                                     (wk * C::BM + (wm * C::FM + i) * 16 + r) * C::kSumPitch +
                                     (wn * C::FN + j) * 16 + 4 * g) = acc[i][j];
    __syncthreads();
    constexpr int kUnits = C::BN / 4;
    for (int u = tid; u < C::BM * kUnits; u += C::kThreads) {
        const int row = u / kUnits, c = u % kUnits * 4;
        if (t.m0 + row >= t.mend)
            break;
        v4f v = *reinterpret_cast<const v4f *>(sums + row * C::kSumPitch + c);
#pragma unroll
        for (int w = 1; w < C::WK; ++w)
            v += *reinterpret_cast<const v4f *>(sums + (w * C::BM + row) * C::kSumPitch + c);
        const int64_t n = t.n0 + c;
        if (n >= a.N)
            continue;
        uint2 b = make_uint2(0, 0);
        if (a.bias)
            b = *reinterpret_cast<const uint2 *>(a.bias + (int64_t)t.e * a.N + n);
        uint2 *o = reinterpret_cast<uint2 *>(a.out + (int64_t)(t.m0 + row) * a.N + n);
        if (a.type == kTypeBf16)
            *o = finish4<kTypeBf16>(v, a.bias != nullptr, b, a.act);
        else
            *o = finish4<kTypeF16>(v, a.bias != nullptr, b, a.act);
    }
}

// ---------------------------------------------------------------------------
// Many rows.  BM x BN outputs per block, WM x WN wavefronts of FM x FN tiles
// of 32 x 32, stages of one block of K (128 bytes of each row) in a ring of
// two LDS buffers filled by direct global->LDS loads; the swizzle of the
// staged rows is gemm::Cfg's.  A lane's scales of four blocks (its FM rows'
// and the weight's) are one dword each, loaded four stages ahead and shifted
// down by a byte per stage.
// ---------------------------------------------------------------------------
template <class C>
struct BigLoads {
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t offA[C::kAInstr], offB[C::kBInstr];

    __device__ __forceinline__ void init(const B128Args &a, const Tile &t, int wave, int lane)
    {
        const int64_t xr = x_base_row(a, t), wr = (int64_t)t.e * a.N + t.n0;
        ra = resource(a.Xq + xr * a.K, (a.rows - xr) * a.K);
        rb = resource(a.CB + wr * a.K, ((int64_t)a.E * a.N - wr) * a.K);
        const int lr = lane / C::kChunks, ls = lane % C::kChunks;
#pragma unroll
        for (int j = 0; j < C::kAInstr; ++j) {
            const int r = (wave * C::kAInstr + j) * C::kRowsPerInstr + lr;
            const int64_t row = source_row(a, t, t.m0 + r) - xr;
            offA[j] = (uint32_t)(row * a.K + ((ls ^ C::swz(r)) << 4));
        }
#pragma unroll
        for (int j = 0; j < C::kBInstr; ++j) {
            const int r = (wave * C::kBInstr + j) * C::kRowsPerInstr + lr;
            const int64_t row = t.n0 + r < a.N ? r : a.N - 1 - t.n0;   // ragged: clamp
            offB[j] = (uint32_t)(row * a.K + ((ls ^ C::swz(r)) << 4));
        }
    }
    __device__ __forceinline__ void issue_one(char *smem, int buf, uint32_t kbyte, int wave,
                                              int j) const
    {
        char *sa = smem + buf * C::kStageBytes;
        char *sb = sa + C::BM * C::ROWB;
        if (j < C::kAInstr)
            gemm::lds_load16(ra, (lds_void *)(sa + (wave * C::kAInstr + j) * 1024), offA[j], kbyte);
        else
            gemm::lds_load16(rb, (lds_void *)(sb + (wave * C::kBInstr + j - C::kAInstr) * 1024),
                             offB[j - C::kAInstr], kbyte);
    }
};

// Keeps the MFMAs on `v` between the side-effecting operations around this
// point: an MFMA is a pure value to the compiler, which otherwise gathers a
// k-step's MFMAs in one run and leaves the loads and reads between two runs.
__device__ __forceinline__ void pin(v16f &v) { asm volatile("" : "+a"(v)); }

// One 64-deep k-step in a fixed issue order: before each MFMA its share of the
// fragment reads of the next k-step and of kNL loads of the stage being
// refilled, so that both run under the MFMAs.
template <class C, int kNL>
__device__ __forceinline__ void kstep(const gemm::Frags8<C> &cur, gemm::Frags8<C> &nxt,
                                      const char *sa, const char *sb, int fo0, int fo1,
                                      v16f (&acc)[C::FM][C::FN], const unsigned (&sx)[C::FM],
                                      unsigned sw, const BigLoads<C> &ld, char *smem, int buf,
                                      uint32_t kbyte, int wave)
{
    constexpr int kReads = C::FM + C::FN, kMfma = C::FM * C::FN;
#pragma unroll
    for (int m = 0; m < kMfma; ++m) {
#pragma unroll
        for (int g = m * kNL / kMfma; g < (m + 1) * kNL / kMfma; ++g)
            ld.issue_one(smem, buf, kbyte, wave, g);
#pragma unroll
        for (int g = (m * kReads + kMfma - 1) / kMfma; g < ((m + 1) * kReads + kMfma - 1) / kMfma; ++g)
            gemm::read_one8<C>(nxt, sa, sb, fo0, fo1, g);
        const int i = m / C::FN, j = m % C::FN;
        pin(acc[i][j]);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(cur.b[j], cur.a[i], acc[i][j],
                                                                    0, 0, 0, sw, 0, sx[i]);
        pin(acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <class C>
__global__ __launch_bounds__(C::kThreads) void k_b128_big(B128Args a)
{
    static_assert(C::ROWB == 128 && C::STAGES == 2, "one block of K per stage");
    static_assert(C::BN / C::WN <= kB128 && kB128 % (C::BN / C::WN) == 0,
                  "a wavefront's columns share a scale row");
    static_assert(C::BM * C::BN * 2 <= C::kLdsBytes, "output tile fits the ring");
    __shared__ __attribute__((aligned(1024))) char smem[C::kLdsBytes];
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    Tile t;
    if (!find_tile<C::BM, C::BN, C::GROUP>(a, lane, t))
        return;
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int numK = (int)((a.K + kB128 - 1) / kB128), full = (int)(a.K / kB128);

    BigLoads<C> ld;
    ld.init(a, t, wave, lane);

    // scales: this lane's rows and its wavefront's columns
    const int64_t pitch = b128_pitch(a.K);
    const int64_t xr = x_base_row(a, t);
    const __amdgpu_buffer_rsrc_t rsx = resource(a.SX + xr * pitch, (a.rows - xr) * pitch);
    const int64_t ws = min(t.n0 + wn * (C::BN / C::WN), a.N - 1) / kB128;
    const __amdgpu_buffer_rsrc_t rsw =
        resource(a.SB + ((int64_t)t.e * scale_rows(a) + ws) * pitch, pitch);
    uint32_t soff[C::FM];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
        soff[i] = (uint32_t)(
            (source_row(a, t, t.m0 + wm * (C::BM / C::WM) + i * 32 + lane % 32) - xr) * pitch);
    unsigned sx[C::FM], sxn[C::FM], sw, swn;
    auto load_scales = [&](unsigned(&x)[C::FM], unsigned &w, int kt) {
        const uint32_t g = (uint32_t)(kt < numK ? kt : numK - 1) / 4 * 4;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            x[i] = buf_load4(rsx, soff[i], g);
        w = buf_load4(rsw, 0, g);
    };

    v16f acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
                acc[i][j][q] = 0;

    const int frow = (lane & 31) * C::ROWB, h = lane >> 5, swz = C::swz(lane & 31);
    int fo0[2], fo1[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        fo0[s] = frow + (((4 * s + h) ^ swz) << 4);
        fo1[s] = frow + (((4 * s + 2 + h) ^ swz) << 4);
    }
    const int aoff = wm * (C::BM / C::WM) * C::ROWB;
    const int boff = C::BM * C::ROWB + wn * (C::BN / C::WN) * C::ROWB;
    auto kbyte = [&](int s) { return (uint32_t)(s < numK ? s : numK - 1) * C::ROWB; };

    load_scales(sx, sw, 0);
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < C::kLoads; ++j)
            ld.issue_one(smem, s, kbyte(s), wave, j);
    wait_vm<C::kLoads>();   // stage 0 (and the scales, loaded before it)
    __builtin_amdgcn_s_barrier();

    // The loop of gemm::mainloop_f8: fragments one k-step ahead, one barrier
    // per stage before its last k-step, under which the stage's buffer is
    // refilled with the stage after the next.
    gemm::Frags8<C> f0, f1;
#pragma unroll
    for (int q = 0; q < C::FM + C::FN; ++q)
        gemm::read_one8<C>(f0, smem + aoff, smem + boff, fo0[0], fo1[0], q);
    for (int kt = 0; kt < full; ++kt) {
        const char *cs = smem + (kt & 1) * C::kStageBytes;
        const char *ns = smem + (kt + 1 < numK ? (kt + 1) & 1 : kt & 1) * C::kStageBytes;
        kstep<C, 0>(f0, f1, cs + aoff, cs + boff, fo0[1], fo1[1], acc, sx, sw, ld, smem, 0, 0, wave);
        wait_vm<0>();   // stage kt + 1 has landed, and the scales on their way
        __builtin_amdgcn_s_barrier();
        if ((kt & 3) == 0)
            load_scales(sxn, swn, kt + 4);
        kstep<C, C::kLoads>(f1, f0, ns + aoff, ns + boff, fo0[0], fo1[0], acc, sx, sw, ld, smem,
                            kt & 1, kbyte(kt + 2), wave);
        const bool next = (kt & 3) == 3;
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
            sx[i] = next ? sxn[i] : sx[i] >> 8;
        sw = next ? swn : sw >> 8;
    }
    if (full < numK) {   // a last block of 64: its first k-step, already in f0
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
            for (int j = 0; j < C::FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    f0.b[j], f0.a[i], acc[i][j], 0, 0, 0, sw, 0, sx[i]);
    }
    wait_vm<0>();      // the tail loads have landed
    __syncthreads();   // and nobody reads the ring any more

    // The finished tile goes out through LDS in whole lines (a lane holds 4
    // columns of one row at a time): 8-byte unit u of row r sits in slot
    // u ^ (r & mask), so that the rows of a tile write without conflicts.
    constexpr int kUnits = C::BN / 4, kMask = kUnits < 32 ? kUnits - 1 : 31;
    const int tl = lane & 31;
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = wn * (C::BN / C::WN) + j * 32 + 8 * q + 4 * h;   // column in the tile
            uint2 b = make_uint2(0, 0);
            if (a.bias) {
                const int64_t n = t.n0 + c < a.N ? t.n0 + c : a.N - 4;
                b = *reinterpret_cast<const uint2 *>(a.bias + (int64_t)t.e * a.N + n);
            }
#pragma unroll
            for (int i = 0; i < C::FM; ++i) {
                const int row = wm * (C::BM / C::WM) + i * 32 + tl;
                const v4f v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                               acc[i][j][4 * q + 3]};
                const uint2 o = a.type == kTypeBf16
                                    ? finish4<kTypeBf16>(v, a.bias != nullptr, b, a.act)
                                    : finish4<kTypeF16>(v, a.bias != nullptr, b, a.act);
                *reinterpret_cast<uint2 *>(smem + row * (C::BN * 2) +
                                           8 * ((c / 4) ^ (row & kMask))) = o;
            }
        }
    }
    __syncthreads();
    constexpr int kPieces = C::BN / 8, kRowsPerPass = C::kThreads / kPieces;
    const int p = tid % kPieces;
#pragma unroll 4
    for (int r = tid / kPieces; r < C::BM; r += kRowsPerPass) {
        uint4 v = *reinterpret_cast<const uint4 *>(smem + r * (C::BN * 2) +
                                                   16 * (p ^ ((r & kMask) >> 1)));
        if (r & 1)
            v = make_uint4(v.z, v.w, v.x, v.y);
        const int64_t n = t.n0 + 8 * p;
        if (t.m0 + r < t.mend && n < a.N)
            *reinterpret_cast<uint4 *>(a.out + (int64_t)(t.m0 + r) * a.N + n) = v;
    }
}

template <class C>
hipError_t launch_tiles(void (*kernel)(B128Args), const B128Args &a, hipStream_t s)
{
    const int64_t ntn = (a.N + C::BN - 1) / C::BN;
    // at most M / BM whole tiles and a ragged one per expert
    const int64_t ntm = a.offsets ? a.M / C::BM + (a.E < a.M ? a.E : a.M) : (a.M + C::BM - 1) / C::BM;
    if (ntm * ntn * C::kThreads > 0xffffffffll)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(ntm * ntn)), dim3(C::kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace b128
}  // namespace llmint8
