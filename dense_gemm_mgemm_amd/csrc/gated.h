// Training form of the gated feed-forward block, FP16 and BF16:
//     G = X Wg, U = X Wu, Z = SiLU(G) * U                       (forward)
//     s = 1 / (1 + e^-G), dU = dZ * G s, dG = dZ * U s (1 + G (1 - s)),
//     dX = dG Wg^T + dU Wu^T, dWg = X^T dG, dWu = X^T dU        (backward)
// Arguments and launchers of its kernels.
#pragma once
#include "common.h"

namespace mgemm {

// Two products side by side (the block's gate and up halves): entry 0 of a
// pair belongs to Wg, entry 1 to Wu.  Equal entries share one matrix.
struct BlockArgs {
    int64_t M, N, K;          // one product's outputs and the contraction of one segment
    const void* A[2];
    int64_t lda;
    const void* B[2];
    int64_t ldb;
    int64_t Mr, Nr;           // readable extents of an M-contiguous A and an N-contiguous B, multiples of 8
    void* C[2];               // forward: G and U (both null: not stored); recomputed backward: dG and dU
    int64_t ldc;
    int batches_m, batches_n; // weights' gradients: 2 along the axis whose operand differs, else 1
    float beta;
    const void* dZ;           // recomputed backward: Mz x Nz, zeros beyond
    int64_t Mz, Nz;
    void* Z;                  // forward
    int64_t ldz;              // of Z or dZ
    float* part;              // split contraction: [tile][range][chunk][thread] f32x4
    int ksplit, nks;          // ranges, and slices per range
};

// Which product: the pair G, U with its epilogue, dX (two segments summed),
// or the two weights' gradients.
enum BlockForm : int { BLOCK_FORWARD = 0, BLOCK_AGAIN = 1, BLOCK_DX = 2, BLOCK_DW = 3 };

struct BlockTile {
    int size;                 // rows and B columns of a tile (forward: half of the columns for each product)
    int ks;                   // ranges of the contraction
};

// Elements of the contraction that a tile takes per slice.
constexpr int slice_of(int size) { return size == 256 ? 32 : 64; }
// Ranges that a request for at most `requested` turns into (whole slices per range).
int block_splits(int64_t slices, int requested);

// b_kc: the pair's B matrices (weights) are contiguous along the contraction.
hipError_t launch_block_forward(const BlockArgs& a, int dtype, bool b_kc, bool again, BlockTile t, hipStream_t s);
hipError_t launch_block_dx(const BlockArgs& a, int dtype, bool b_kc, BlockTile t, hipStream_t s);
hipError_t launch_block_dw(const BlockArgs& a, int dtype, BlockTile t, hipStream_t s);

// dX and the weights' gradients in one launch, both in 128x128 tiles, and
// one more for the sums of what is split.
hipError_t launch_block_pair(const BlockArgs& x, const BlockArgs& w, int dtype, bool b_kc, int xks, int wks,
                             hipStream_t s);

// dG and dU from G, U and dZ (M x N): Mo x No of them, zeros past M x N, in
// rows of ldd elements (No and ldd multiples of 8, 16-byte aligned).
hipError_t launch_gated_grad(int64_t M, int64_t N, int64_t Mo, int64_t No, const void* G, const void* U, int64_t ldg, const void* dZ,
                             int64_t lddz, void* dG, void* dU, int64_t ldd, int dtype, hipStream_t s);
// Copies up to three 16-bit matrices to rows of ldd elements (a multiple of 8,
// 16-byte aligned), zeros past their columns and in the rows up to rows_out.
struct Repack {
    const void* src[3];
    void* dst[3];
    int64_t rows[3], cols[3], lds[3], ldd[3], rows_out[3];
    int n;
};
hipError_t launch_repack(const Repack& r, hipStream_t s);

}  // namespace mgemm
