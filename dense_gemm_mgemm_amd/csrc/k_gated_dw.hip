// dWg = X^T dG and dWu = X^T dU (or their transposes) in one grid (see
// gated_tile.h): A is contiguous along the outputs' rows, B along their columns.
//
// Measured (kernels alone): 1024 x 12288 x 4096 BF16 209 to 252 us (1536 workgroups,
// six to a CU, of 3.8 us to the first MFMA, 31 in the loop of 32 slices and 6.8
// for 128 KiB of outputs, 33 MB at once on all CUs: HBM's rate); 1024 x 1536 x
// 4096 34 us.  Both operands are read transposed: the loop is bound by LDS.
#include "gated_tile.h"

namespace mgemm {
namespace {

template <int DT>
hipError_t by_tile(const BlockArgs& a, BlockTile t, hipStream_t s) {
    return t.size == 128 ? launch_block<DT, BLOCK_DW, 128, true, false>(a, t.ks, s)
                         : launch_block<DT, BLOCK_DW, 256, true, false>(a, t.ks, s);
}

}  // namespace

hipError_t launch_block_dw(const BlockArgs& a, int dtype, BlockTile t, hipStream_t s) {
    return dtype == F16 ? by_tile<F16>(a, t, s) : by_tile<BF16>(a, t, s);
}

}  // namespace mgemm
