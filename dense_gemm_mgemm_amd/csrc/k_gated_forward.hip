// G = X Wg and U = X Wu in one tile (see gated_tile.h), with the forward
// epilogue (Z, G, U) or the backward's (dG and dU from G, U computed again, and
// dZ).
//
// Measured: 1024 x 1536 x 4096 BF16, weights in x out, 32 to 34 us (0.78 PFLOP/s): 192
// workgroups of 128 tiles (256 tiles in 4 ranges 45), of which 30 in the tile
// loop, bound by LDS (the weights' transposed reads move half the bytes per
// clock).  777 x 1000 x 1001 FP16 with odd strides 20.3: 5.6 for the copies, 12.7
// for the product, of which 6.6 in the loop and the rest the first load and the
// stores.
#include "gated_tile.h"

namespace mgemm {
namespace {

template <int DT, int FORM, bool BKC>
hipError_t by_tile(const BlockArgs& a, BlockTile t, hipStream_t s) {
    return t.size == 128 ? launch_block<DT, FORM, 128, false, BKC>(a, t.ks, s)
                         : launch_block<DT, FORM, 256, false, BKC>(a, t.ks, s);
}
template <int DT, int FORM>
hipError_t by_layout(const BlockArgs& a, bool b_kc, BlockTile t, hipStream_t s) {
    return b_kc ? by_tile<DT, FORM, true>(a, t, s) : by_tile<DT, FORM, false>(a, t, s);
}

}  // namespace

hipError_t launch_block_forward(const BlockArgs& a, int dtype, bool b_kc, bool again, BlockTile t, hipStream_t s) {
    if (dtype == F16)
        return again ? by_layout<F16, BLOCK_AGAIN>(a, b_kc, t, s) : by_layout<F16, BLOCK_FORWARD>(a, b_kc, t, s);
    return again ? by_layout<BF16, BLOCK_AGAIN>(a, b_kc, t, s) : by_layout<BF16, BLOCK_FORWARD>(a, b_kc, t, s);
}

}  // namespace mgemm
