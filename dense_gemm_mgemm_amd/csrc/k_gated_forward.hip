// G = X Wg and U = X Wu in one tile (see gated_tile.h),
// with the forward epilogue (Z, G, U) or the backward's (dG and dU from G, U
// computed again, and dZ).
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
