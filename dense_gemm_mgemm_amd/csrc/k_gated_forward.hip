// G = X Wg and U = X Wu in one tile of 96 columns of each (see gated_tile.h),
// with the forward epilogue (Z, G, U) or the backward's (dG and dU from G, U
// computed again, and dZ).
#include "gated_tile.h"

namespace mgemm {
namespace {

template <int DT, int FORM>
hipError_t by_tile(const BlockArgs& a, bool b_kc, BlockTile t, hipStream_t s) {
    if (b_kc)
        return t.bm == 256 ? launch_block<DT, FORM, 256, 192, false, true>(a, t.ks, s)
                           : launch_block<DT, FORM, 128, 192, false, true>(a, t.ks, s);
    return t.bm == 256 ? launch_block<DT, FORM, 256, 192, false, false>(a, t.ks, s)
                       : launch_block<DT, FORM, 128, 192, false, false>(a, t.ks, s);
}

}  // namespace

hipError_t launch_block_forward(const BlockArgs& a, int dtype, bool b_kc, bool again, BlockTile t, hipStream_t s) {
    if (dtype == F16)
        return again ? by_tile<F16, BLOCK_AGAIN>(a, b_kc, t, s) : by_tile<F16, BLOCK_FORWARD>(a, b_kc, t, s);
    return again ? by_tile<BF16, BLOCK_AGAIN>(a, b_kc, t, s) : by_tile<BF16, BLOCK_FORWARD>(a, b_kc, t, s);
}

}  // namespace mgemm
