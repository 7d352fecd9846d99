// dX and the weights' gradients of a small block in one launch: each alone
// leaves CUs idle, and a launch of its own costs what its few slices do
// (333 x 1004 x 515 FP16, computed again: 9.4 us and 2.8 for the sums,
// against 5.8, 2.9 and 7.8 in three launches with their gaps; the whole pass 31.8
// against 37.6).
#include "gated_tile.h"

namespace mgemm {
namespace {

constexpr int PT = 128;                         // tile rows and columns of both products

template <int DT, bool BKC>
__global__ __launch_bounds__(NT, 1) void k_block_pair(BlockArgs x, BlockArgs w, int nx) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int bid = blockIdx.x;
    if (bid < nx) block_body<DT, BLOCK_DX, PT, false, BKC, STORE_EITHER>(x, bid, nx, smem);
    else block_body<DT, BLOCK_DW, PT, true, false, STORE_EITHER>(w, bid - nx, gridDim.x - nx, smem);
}

template <int DT>
__global__ __launch_bounds__(NT) void k_block_pair_reduce(BlockArgs x, BlockArgs w, int nx) {
    const int bid = blockIdx.x;
    if (bid < nx) reduce_body<DT, BLOCK_DX, PT>(x, bid, nx);
    else reduce_body<DT, BLOCK_DW, PT>(w, bid - nx, gridDim.x - nx);
}

template <int DT, bool BKC>
hipError_t launch(BlockArgs x, BlockArgs w, int xks, int wks, hipStream_t s) {
    using G = Cfg<BLOCK_DX, PT>;
    const int64_t nx = set_ranges<BLOCK_DX, PT>(x, xks), nw = set_ranges<BLOCK_DW, PT>(w, wks);
    // The partial sums of dW lie behind those of dX.
    if (x.ksplit > 1) w.part += nx * (PT * PT);
    auto kern = k_block_pair<DT, BKC>;
    static bool done[MAX_DEVICES] = {};
    if (hipError_t e = set_lds_limit_once((const void*)kern, G::LDS, done); e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((unsigned)(nx + nw)), dim3(NT), G::LDS, s, x, w, (int)nx);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const int64_t rx = x.ksplit > 1 ? nx / x.ksplit * reduce_chunks<BLOCK_DX, PT>() : 0;
    const int64_t rw = w.ksplit > 1 ? nw / w.ksplit * reduce_chunks<BLOCK_DW, PT>() : 0;
    if (rx + rw == 0) return hipSuccess;
    hipLaunchKernelGGL(k_block_pair_reduce<DT>, dim3((unsigned)(rx + rw)), dim3(NT), 0, s, x, w, (int)rx);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_block_pair(const BlockArgs& x, const BlockArgs& w, int dtype, bool b_kc, int xks, int wks,
                             hipStream_t s) {
    if (dtype == F16) return b_kc ? launch<F16, true>(x, w, xks, wks, s) : launch<F16, false>(x, w, xks, wks, s);
    return b_kc ? launch<BF16, true>(x, w, xks, wks, s) : launch<BF16, false>(x, w, xks, wks, s);
}

}  // namespace mgemm
