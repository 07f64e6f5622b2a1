// b128_gemm.hip -- instantiations of the block-scaled FP8 product
// (b128_gemm.h) and the choice among them.
#include "b128_gemm.h"

namespace llmint8 {

using Small16 = b128::SmallCfg<16, 16, 1, 1, 4, 4>;
using Small16x32 = b128::SmallCfg<16, 32, 1, 1, 4, 3>;
using Small32 = b128::SmallCfg<32, 32, 1, 1, 4, 2>;
using Small64 = b128::SmallCfg<64, 64, 2, 2, 1, 2>;
using Big64 = b128::BigCfg<64, 128, 1, 4, 3, 4>;
using Big128 = b128::BigCfg<128, 128, 2, 2, 2, 4>;
using Big256 = b128::BigCfg<256, 256, 2, 2, 2, 4>;

namespace {

// The tile and the parts of K, by an estimate in microseconds that follows
// what the sweeps on MI355X showed.  A block reads (BM + BN) * K bytes, at 52
// KB/us per compute unit whatever its shape (the 13 TB/s that all of them
// draw from L2 together); only 256 x 256 reaches the matrix cores' pace, 1.5
// us per block of K.  The weight comes from HBM once at 5 TB/s.  A block costs
// `fixed` besides (first loads, output), less where several are resident; a
// split of K costs a second launch and its partial sums, written and read.
// Measured (us; the estimate's choice first): 300 x 2048 x 8192 128 x 128 12.8,
// 64 x 128 15.4, 64 x 64 24.7; 256 x 4096 x 4096 64 x 64 14.8, 64 x 128 17.1, 128 x 128
// 20.3; 64 x 16384 x 4096 64 x 128 in 8 parts 20.9, 128 x 128 in 8 23.4, 32 x 32 whole
// 32.1; 512 x 16384 x 4096 128 x 128 in 4 parts 51.2, 64 x 128 whole 57.0; 1 x 4096
// x 4096 16 x 16 5.9, 16 x 32 6.5; 64 experts with one row, K = 2048, N = 1024: 16 x 32
// 34.7, 16 x 16 44.6.
struct Shape {
    int bm, bn;
    double fixed, per_block;   // per_block: us per block of K if not bound by reading
    hipError_t (*launch)(const B128Args &, hipStream_t);
};
const Shape kShapes[kB128Paths] = {
    {16, 16, 0.8, 0.0, b128::launch_small<Small16>},
    {16, 32, 0.8, 0.0, b128::launch_small<Small16x32>},
    {32, 32, 0.8, 0.0, b128::launch_small<Small32>},
    {64, 64, 1.5, 0.0, b128::launch_small<Small64>},
    {64, 128, 1.0, 0.0, b128::launch_big<Big64>},
    {128, 128, 1.0, 0.0, b128::launch_big<Big128>},
    {256, 256, 4.0, 1.5, b128::launch_big<Big256>},
};
constexpr double kCuRate = 52e3, kHbmRate = 5e6;   // bytes per us
constexpr int kCUs = 256;
constexpr int64_t kMostParts = (int64_t)128 << 20;   // bytes of partial sums

struct Plan {
    const Shape *shape;
    int nparts, per;   // parts of K, blocks of K in each
};

// path: 0, or the number of the only shape to consider (1 ..); parts: 0, or the
// only number of parts (fewer if K has fewer groups of four blocks).
Plan choose(int64_t M, int64_t K, int64_t N, int64_t E, bool grouped, int path, int only)
{
    const int64_t nblk = (K + kB128 - 1) / kB128, used = E < M ? E : M;
    const double hbm = (double)used * N * K / kHbmRate;
    Plan best{&kShapes[0], 1, (int)nblk};
    double least = 1e300;
    for (int i = 0; i < kB128Paths; ++i) {
        const Shape &s = kShapes[i];
        if (path && path != i + 1)
            continue;
        // rows of tiles: of a grouped product, each expert's last one is half full on average
        double ntm = (double)((M + s.bm - 1) / s.bm);
        if (grouped) {
            ntm = (double)M / s.bm + 0.5 * used;
            ntm = ntm < used ? used : ntm;
        }
        const double tiles = ntm * ((N + s.bn - 1) / s.bn);
        for (int parts = only ? only : 1; parts <= 8; parts *= 2) {
            if (parts > 1 && !only &&
                (grouped || nblk < 8 * parts || parts * M * N * 4 > kMostParts))
                break;
            const int per = (int)((nblk + parts - 1) / parts + 3) / 4 * 4;   // whole dwords of scales
            const int n = (int)((nblk + per - 1) / per);
            const double read = (double)(s.bm + s.bn) * per * kB128 / kCuRate;
            const double one = s.fixed + (read > per * s.per_block ? read : per * s.per_block);
            const double rounds = __builtin_ceil(tiles * n / kCUs);
            double t = rounds * one;
            t = t < hbm ? hbm : t;
            if (n > 1)
                t += 3.0 + 2.0 * n * M * N * 4 / kHbmRate;
            if (t < least) {
                least = t;
                best = Plan{&s, n, per};
            }
            if (only)
                break;
        }
    }
    return best;
}

}  // namespace

size_t b128_workspace_bytes(int64_t T, int64_t K, int64_t N, int path, int parts)
{
    const Plan p = choose(T, K, N, 1, false, path, parts);
    return p.nparts > 1 ? (size_t)p.nparts * T * N * 4 : 0;
}

hipError_t launch_matmul_b128(const B128Args &args, void *ws, int path, int parts, hipStream_t s)
{
    const Plan p = choose(args.M, args.K, args.N, args.E, args.offsets != nullptr, path, parts);
    B128Args a = args;
    if (p.nparts > 1) {
        a.nparts = p.nparts;
        a.per = p.per;
        a.parts = static_cast<float *>(ws);
    }
    const hipError_t e = p.shape->launch(a, s);
    return e == hipSuccess && p.nparts > 1 ? b128::launch_sum(a, s) : e;
}

}  // namespace llmint8
