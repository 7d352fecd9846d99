// dX = dG Wg^T + dU Wu^T as one product over two segments (see gated_tile.h).
//
// Measured (kernels alone): 1024 x 12288 x 4096 BF16, weights in x out, 178 to 197
// us and 13 for the sum of 4 ranges (206 GFLOP: 1.0 to 1.1 PFLOP/s, the rate of a
// large library product, which is the chip's power limit); 1024 x 1536 x 4096,
// weights out x in, 31 us on 256 workgroups of 128 tiles.
#include "gated_tile.h"

namespace mgemm {
namespace {

template <int DT, bool BKC>
hipError_t by_tile(const BlockArgs& a, BlockTile t, hipStream_t s) {
    return t.size == 128 ? launch_block<DT, BLOCK_DX, 128, false, BKC>(a, t.ks, s)
                         : launch_block<DT, BLOCK_DX, 256, false, BKC>(a, t.ks, s);
}

}  // namespace

hipError_t launch_block_dx(const BlockArgs& a, int dtype, bool b_kc, BlockTile t, hipStream_t s) {
    if (dtype == F16) return b_kc ? by_tile<F16, true>(a, t, s) : by_tile<F16, false>(a, t, s);
    return b_kc ? by_tile<BF16, true>(a, t, s) : by_tile<BF16, false>(a, t, s);
}

}  // namespace mgemm
