// b128_gemm.hip -- instantiations of the block-scaled FP8 product
// (b128_gemm.h) and the choice among them.
#include "b128_gemm.h"

namespace llmint8 {

using Rows16 = b128::SmallCfg<16, 16, 1, 1, 4, 4>;
using Rows32 = b128::SmallCfg<32, 64, 1, 2, 2, 3>;
using Rows64 = b128::SmallCfg<64, 64, 2, 2, 1, 2>;
using Big128 = b128::BigCfg<128, 128, 2, 2, 4, 4>;
using Big256 = b128::BigCfg<256, 256, 2, 2, 2, 4>;

size_t b128_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }


hipError_t launch_matmul_b128(const B128Args &a, void *, hipStream_t s)
{
    const int64_t rows = (a.M + a.E - 1) / a.E;   // per expert
    if (rows <= 16)
        return b128::launch_small<Rows16>(a, s);
    if (rows <= 32)
        return b128::launch_small<Rows32>(a, s);
    if (rows <= 64)
        return b128::launch_small<Rows64>(a, s);
    if (rows <= 512)
        return b128::launch_big<Big128>(a, s);
    return b128::launch_big<Big256>(a, s);
}

}  // namespace llmint8
