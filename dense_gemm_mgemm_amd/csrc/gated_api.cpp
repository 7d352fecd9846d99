// Entry points of the gated block's training form: argument checks, the
// workspace's layout, tile and split choice, and the order of launches.  See
// include/mgemm.h for the contracts.
#include <hip/hip_runtime.h>

#include "gated.h"
#include "host.h"

using namespace mgemm_host;

namespace {

using mgemm::BlockArgs;
using mgemm::BlockForm;
using mgemm::BlockTile;

constexpr int64_t LIM = (int64_t)1 << 60;

int64_t max1(int64_t x) { return x > 1 ? x : 1; }
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
bool aligned(const void* p) { return ((uintptr_t)p & 15) == 0; }
mgemm_status_t status(hipError_t e) { return e == hipSuccess ? MGEMM_SUCCESS : MGEMM_ERR_HIP; }
bool valid_matrix(int64_t rows, int64_t cols, int64_t ld) { return ld >= max1(cols) && (rows == 0 || ld <= LIM / rows); }

// What one call reads, where its copies and gradients lie in the workspace.
struct Plan {
    bool col;                         // weights stored out x in
    int64_t M, N, K;
    bool copy_x, copy_w;
    int64_t w_rows, w_cols;           // the stored weights' shape
    int64_t x_at, wg_at, wu_at;       // byte offsets of the copies
    int64_t dg_at, du_at;             // of dG and dU,
    int64_t d_rows, d_cols;           //   d_rows x d_cols each, packed
    int64_t bytes;                    // the whole workspace, with room to align its start
};

constexpr int64_t ALIGN = 256;
// Copies are padded with zeros to whole slices of the matrix kernels, and dG
// and dU along an axis that meets a copy: a contraction of two padded operands
// runs over the padded length and has no tail, which costs a workgroup 1.5 to
// 3 us (ordinary loads that nothing overlaps).
constexpr int64_t SLICE = 64;

// The matrix kernels read rows of 16-byte chunks: a stride that is a multiple
// of 8 and an aligned base, and where a row runs along an output axis (not
// along the contraction, whose tail is read element by element) a length that
// is a multiple of 8 as well.  Anything else is copied.
Plan make_plan(mgemm_layout_t layout, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const void* Wg,
               const void* Wu, int64_t ldw, bool forward, bool again, bool dx, bool dw) {
    Plan p{};
    p.col = layout == MGEMM_COL_MAJOR;
    p.M = M; p.N = N; p.K = K;
    p.w_rows = p.col ? N : K;
    p.w_cols = p.col ? K : N;
    const bool uses_x = forward || again || dw, uses_w = forward || again || dx;
    p.copy_x = uses_x && (ldx % 8 != 0 || !aligned(X) || (dw && K % 8 != 0));
    const bool w_whole = p.col ? dx && K % 8 != 0 : (forward || again) && N % 8 != 0;
    p.copy_w = uses_w && (ldw % 8 != 0 || !aligned(Wg) || !aligned(Wu) || w_whole);
    int64_t at = 0;
    auto take = [&](int64_t rows, int64_t cols) {
        const int64_t here = at;
        at += up(rows * cols * 2, ALIGN);
        return here;
    };
    if (p.copy_x) p.x_at = take(up(M, SLICE), up(K, SLICE));
    if (p.copy_w) {
        p.wg_at = take(up(p.w_rows, SLICE), up(p.w_cols, SLICE));
        p.wu_at = take(up(p.w_rows, SLICE), up(p.w_cols, SLICE));
    }
    p.d_rows = p.copy_x ? up(M, SLICE) : M;
    p.d_cols = up(N, p.copy_w ? SLICE : 8);
    if (!forward) {
        p.dg_at = take(p.d_rows, p.d_cols);
        p.du_at = take(p.d_rows, p.d_cols);
    }
    p.bytes = at > 0 ? at + ALIGN : 0;
    return p;
}

// One product's workgroups in tiles of one size and split.
struct Grid {
    BlockTile tile;
    int64_t tiles;
    int64_t wgs;            // tiles x ranges
    int64_t part_bytes;     // of the partial sums (0: whole contractions)
    double wg_us;           // one workgroup
    double sum_us;          // the second phase
    double us;              // the launches
};

// Predicted times (microseconds).  A workgroup takes 0.45 us per 64 elements of
// the contraction in a 128 tile and 1.45 in a 256 tile, and 3.6 or 7 us from
// its launch to its first MFMA and through its outputs; a CU holds one (the ring
// fills its LDS).  A split adds a launch, 0.45 us per range (one thread
// adds them in turn) and its partial sums at 4.8 TB/s.
// Fitted to 45 blocks, 24 x 30 x 161 to 1024 x 12288 x 4096, each product
// timed with both tiles in 1 to 16 ranges; by it the choice is 1% slower than
// the fastest of them in the mean, 4.5 us at worst.  (256 x 192, 128 x 256 and
// 128 x 192 tiles were built and timed too: the best in 6 of 73 products, by
// 10% at most, and are gone.)
Grid grid_of(int num_cu, BlockForm form, const BlockArgs& a, int size, int requested) {
    const bool dual = form == mgemm::BLOCK_FORWARD || form == mgemm::BLOCK_AGAIN;
    const int out = dual ? size / 2 : size, slice = mgemm::slice_of(size);
    const int64_t cus = num_cu > 0 ? num_cu : 256;
    const int64_t slices = a.K / slice * (form == mgemm::BLOCK_DX ? 2 : 1);
    Grid g{};
    g.tile = BlockTile{size, mgemm::block_splits(slices, requested)};
    g.tiles = (a.M + size - 1) / size * a.batches_m * ((a.N + out - 1) / out * a.batches_n);
    g.wgs = g.tiles * g.tile.ks;
    const int64_t per = (slices + g.tile.ks - 1) / g.tile.ks;
    g.wg_us = (double)per * slice / 64 * (size == 256 ? 1.45 : 0.45) + (size == 256 ? 7.0 : 3.6);
    if (g.tile.ks > 1) {
        g.part_bytes = g.wgs * size * size * 4;
        g.sum_us = 3.0 + 0.45 * g.tile.ks + (double)g.part_bytes / 4.8e6;
    }
    // Few rounds of workgroups end together; many even out.
    const double rounds = g.wgs <= 4 * cus ? (double)((g.wgs + cus - 1) / cus) : (double)g.wgs / cus;
    g.us = rounds * g.wg_us + g.sum_us;
    return g;
}

// The grids that a product may run as (those of its forced tile), a few splits
// of each size: the choice is made in every call, on the host.
struct Grids {
    Grid g[2 * 12];
    int n = 0;
};
Grids grids_of(mgemm_handle_t h, BlockForm form, const BlockArgs& a) {
    static constexpr int SPLITS[12] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 24, 32};
    const auto& forced = h->gated_tile[form == mgemm::BLOCK_DX ? 1 : form == mgemm::BLOCK_DW ? 2 : 0];
    Grids out;
    for (int size : {256, 128}) {
        if (forced.size != 0 && forced.size != size) continue;
        int last = 0;
        for (int req : SPLITS) {
            if (forced.ksplit != 0) req = forced.ksplit;
            const Grid g = grid_of(h->num_cu, form, a, size, req);
            if (g.tile.ks <= last) continue;
            last = g.tile.ks;
            if (g.part_bytes <= h->ws.part_bytes) out.g[out.n++] = g;
        }
    }
    return out;
}

// The fastest by prediction; wgs 0: none fits the workspace (a forced split).
Grid fastest(const Grids& all) {
    Grid best{};
    for (int i = 0; i < all.n; ++i)
        if (best.wgs == 0 || all.g[i].us < best.us) best = all.g[i];
    return best;
}

// Whether dX and the weights' gradients run as one launch of 128 tiles, and
// then in which splits: where both together fill the CUs at most twice, the
// launch lasts as long as the longer of its workgroups and not as the sum of
// two launches (333 x 1004 x 515 FP16 computed again: 31.8 us against 37.6).
bool choose_pair(mgemm_handle_t h, const Grids& x, const Grids& w, Grid& xg, Grid& wg) {
    const int64_t cus = h->num_cu > 0 ? h->num_cu : 256;
    double best = xg.us + wg.us;
    bool pair = false;
    for (int i = 0; i < x.n; ++i) {
        const Grid& a = x.g[i];
        if (a.tile.size != 128 || a.wgs > 2 * cus) continue;
        for (int j = 0; j < w.n; ++j) {
            const Grid& b = w.g[j];
            if (b.tile.size != 128 || a.wgs + b.wgs > 2 * cus || a.part_bytes + b.part_bytes > h->ws.part_bytes)
                continue;
            const double longer = a.wg_us > b.wg_us ? a.wg_us : b.wg_us;
            const double shared = (a.wgs * a.wg_us + b.wgs * b.wg_us) / cus + (a.wgs + b.wgs > cus ? longer / 2 : 0.0);
            const double us = (longer > shared ? longer : shared) + (a.sum_us > b.sum_us ? a.sum_us : b.sum_us);
            if (us < best) {
                best = us;
                pair = true;
                xg = a;
                wg = b;
            }
        }
    }
    return pair;
}

// Whether the grids and slice counts of these sizes stay within 32 bits.
bool fits(int64_t M, int64_t N, int64_t K) {
    const int64_t most = (int64_t)0x7fffffff / 64;
    auto tiles = [](int64_t m, int64_t n) { return ((m + 127) / 128) * 2 * ((n + 63) / 64); };
    return M / 32 < 0x3fffffff && N / 32 < 0x3fffffff && K / 32 < 0x3fffffff && (M + 127) / 128 < most &&
           (N + 63) / 64 < most && (K + 63) / 64 < most && tiles(M, N) < most && tiles(M, K) < most &&
           tiles(K, N) < most && tiles(N, K) < most;
}

// Outputs M x N (two of them along an axis with two batches) of a contraction over K.
BlockArgs base_args(const mgemm::Workspace& ws, int64_t M, int64_t N, int64_t K) {
    BlockArgs a{};
    a.M = M; a.N = N; a.K = K;
    a.Mr = up(M, 8); a.Nr = up(N, 8);
    a.batches_m = a.batches_n = 1;
    a.part = (float*)ws.part;
    return a;
}

struct Operands {
    const void *X, *Wg, *Wu;
    int64_t ldx, ldw;
};

// Copies what has to be copied, and says where the operands are from then on.
mgemm_status_t lay_out(const Plan& p, char* work, Operands& o, hipStream_t s) {
    mgemm::Repack r{};
    auto add = [&](const void*& src, int64_t rows, int64_t cols, int64_t ld, int64_t at) {
        r.src[r.n] = src;
        r.dst[r.n] = work + at;
        r.rows[r.n] = rows; r.cols[r.n] = cols; r.lds[r.n] = ld; r.ldd[r.n] = up(cols, SLICE);
        r.rows_out[r.n] = up(rows, SLICE);
        ++r.n;
        src = work + at;
    };
    if (p.copy_x) {
        add(o.X, p.M, p.K, o.ldx, p.x_at);
        o.ldx = up(p.K, SLICE);
    }
    if (p.copy_w) {
        add(o.Wg, p.w_rows, p.w_cols, o.ldw, p.wg_at);
        add(o.Wu, p.w_rows, p.w_cols, o.ldw, p.wu_at);
        o.ldw = up(p.w_cols, SLICE);
    }
    return r.n > 0 ? status(mgemm::launch_repack(r, s)) : MGEMM_SUCCESS;
}

// C (rows x cols, 16-bit) = beta * C.
mgemm_status_t scale(mgemm_handle_t h, void* C, int64_t rows, int64_t cols, int64_t ld, float beta, int dtype,
                     hipStream_t s) {
    if (C == nullptr || rows == 0 || cols == 0) return MGEMM_SUCCESS;
    Problem q{};
    q.M = rows; q.N = cols;
    q.beta = beta;
    q.C = C; q.ldc = ld;
    q.dtype = dtype;
    q.num_cu = h->num_cu;
    q.epilogue = mgemm::EPI_NONE;
    return status(mgemm::launch_scale(q, s));
}

mgemm_status_t check_common(mgemm_layout_t layout, int64_t M, int64_t N, int64_t K, int64_t ldx, int64_t ldw,
                            mgemm_dtype_t dtype) {
    if (layout != MGEMM_ROW_MAJOR && layout != MGEMM_COL_MAJOR) return MGEMM_ERR_INVALID_ARG;
    if (dtype != MGEMM_F32 && dtype != MGEMM_F16 && dtype != MGEMM_BF16) return MGEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || M > LIM || N > LIM || K > LIM) return MGEMM_ERR_INVALID_ARG;
    const bool col = layout == MGEMM_COL_MAJOR;
    if (!valid_matrix(M, K, ldx) || !valid_matrix(col ? N : K, col ? K : N, ldw)) return MGEMM_ERR_INVALID_ARG;
    if (dtype == MGEMM_F32) return MGEMM_ERR_UNSUPPORTED;
    // The workspace's byte counts are sums of a few products of two sizes.
    const int64_t lim = LIM / 8;
    if ((N > 0 && M > lim / (N + 8)) || (K > 0 && M > lim / (K + 8)) || (K > 0 && N > lim / (K + 8)) ||
        (N > 0 && K > lim / (N + 8)))
        return MGEMM_ERR_INVALID_ARG;
    return MGEMM_SUCCESS;
}

// The workspace's start (aligned), or null when it is too small.
mgemm_status_t check_work(const Plan& p, void* work, int64_t bytes, char** out) {
    *out = nullptr;
    if (p.bytes == 0) return MGEMM_SUCCESS;
    if (work == nullptr || bytes < p.bytes) return MGEMM_ERR_INVALID_ARG;
    *out = (char*)up((int64_t)(uintptr_t)work, ALIGN);
    return MGEMM_SUCCESS;
}

}  // namespace

namespace mgemm {

int block_splits(int64_t slices, int requested) {
    if (requested <= 1 || slices < 2) return 1;
    const int64_t ks = requested < slices ? requested : slices, nks = (slices + ks - 1) / ks;
    return (int)((slices + nks - 1) / nks);
}

}  // namespace mgemm

extern "C" {

mgemm_status_t mgemm_gated_workspace(mgemm_layout_t layoutW, int64_t M, int64_t N, int64_t K, const void* X,
                                     int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, mgemm_dtype_t dtype,
                                     int32_t backward, int32_t stored, int64_t* bytes) {
    if (!bytes) return MGEMM_ERR_INVALID_ARG;
    const mgemm_status_t st = check_common(layoutW, M, N, K, ldx, ldw, dtype);
    if (st != MGEMM_SUCCESS) return st;
    const bool b = backward != 0;
    *bytes = M == 0 || N == 0 || K == 0
                 ? 0
                 : make_plan(layoutW, M, N, K, X, ldx, Wg, Wu, ldw, !b, b && stored == 0, b, b).bytes;
    return MGEMM_SUCCESS;
}

mgemm_status_t mgemm_set_gated_tile(mgemm_handle_t h, int32_t product, int32_t size, int32_t ksplit) {
    if (!h || product < 0 || product > 2 || ksplit < 0 || ksplit > MGEMM_MAX_KSPLIT) return MGEMM_ERR_INVALID_ARG;
    if (size != 0 && size != 128 && size != 256) return MGEMM_ERR_INVALID_ARG;
    h->gated_tile[product] = mgemm_host::GatedTile{size, ksplit};
    return MGEMM_SUCCESS;
}

mgemm_status_t mgemm_gated_forward(mgemm_handle_t h, mgemm_layout_t layoutW, int64_t M, int64_t N, int64_t K,
                                   const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t ldw, void* Z,
                                   int64_t ldz, void* G, void* U, int64_t ldg, mgemm_dtype_t dtype, void* work,
                                   int64_t work_bytes, hipStream_t stream) {
    if (!h) return MGEMM_ERR_INVALID_ARG;
    if (const mgemm_status_t st = check_common(layoutW, M, N, K, ldx, ldw, dtype); st != MGEMM_SUCCESS) return st;
    if (!valid_matrix(M, N, ldz) || (G == nullptr) != (U == nullptr) || (G && !valid_matrix(M, N, ldg)))
        return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MGEMM_SUCCESS;
    if (!Z) return MGEMM_ERR_INVALID_ARG;
    if (K == 0) {                                     // G = U = Z = 0
        mgemm_status_t st = scale(h, Z, M, N, ldz, 0.0f, (int)dtype, stream);
        if (st == MGEMM_SUCCESS) st = scale(h, G, M, N, ldg, 0.0f, (int)dtype, stream);
        if (st == MGEMM_SUCCESS) st = scale(h, U, M, N, ldg, 0.0f, (int)dtype, stream);
        return st;
    }
    if (!X || !Wg || !Wu) return MGEMM_ERR_INVALID_ARG;
    if (!fits(M, N, K)) return MGEMM_ERR_UNSUPPORTED;
    const Plan p = make_plan(layoutW, M, N, K, X, ldx, Wg, Wu, ldw, true, false, false, false);
    char* w;
    if (const mgemm_status_t st = check_work(p, work, work_bytes, &w); st != MGEMM_SUCCESS) return st;
    BlockArgs a = base_args(h->ws, M, N, p.copy_x && p.copy_w ? up(K, SLICE) : K);
    const Grid g = fastest(grids_of(h, mgemm::BLOCK_FORWARD, a));
    if (g.wgs == 0) return MGEMM_ERR_UNSUPPORTED;
    Operands o{X, Wg, Wu, ldx, ldw};
    if (const mgemm_status_t st = lay_out(p, w, o, stream); st != MGEMM_SUCCESS) return st;
    a.A[0] = a.A[1] = o.X; a.lda = o.ldx;
    a.B[0] = o.Wg; a.B[1] = o.Wu; a.ldb = o.ldw;
    a.Z = Z; a.ldz = ldz;
    a.C[0] = G; a.C[1] = U; a.ldc = ldg;
    return status(mgemm::launch_block_forward(a, (int)dtype, p.col, false, g.tile, stream));
}

mgemm_status_t mgemm_gated_backward(mgemm_handle_t h, mgemm_layout_t layoutW, int64_t M, int64_t N, int64_t K,
                                    const void* X, int64_t ldx, const void* Wg, const void* Wu, int64_t ldw,
                                    const void* G, const void* U, int64_t ldg, const void* dZ, int64_t lddz, void* dX,
                                    int64_t lddx, void* dWg, void* dWu, int64_t lddw, float beta, mgemm_dtype_t dtype,
                                    void* work, int64_t work_bytes, hipStream_t stream) {
    if (!h) return MGEMM_ERR_INVALID_ARG;
    if (const mgemm_status_t st = check_common(layoutW, M, N, K, ldx, ldw, dtype); st != MGEMM_SUCCESS) return st;
    const bool col = layoutW == MGEMM_COL_MAJOR, again = G == nullptr;
    if ((G == nullptr) != (U == nullptr) || (dWg == nullptr) != (dWu == nullptr)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_matrix(M, N, lddz) || (G && !valid_matrix(M, N, ldg)) || (dX && !valid_matrix(M, K, lddx)) ||
        (dWg && !valid_matrix(col ? N : K, col ? K : N, lddw)))
        return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0 || K == 0) {                 // no terms: dX = 0, dW = beta * dW
        const int64_t rows = col ? N : K, cols = col ? K : N;
        mgemm_status_t st = scale(h, dX, M, K, lddx, 0.0f, (int)dtype, stream);
        if (st == MGEMM_SUCCESS) st = scale(h, dWg, rows, cols, lddw, beta, (int)dtype, stream);
        if (st == MGEMM_SUCCESS) st = scale(h, dWu, rows, cols, lddw, beta, (int)dtype, stream);
        return st;
    }
    if (!dX && !dWg) return MGEMM_SUCCESS;
    if (!dZ || ((again || dWg) && !X) || ((again || dX) && (!Wg || !Wu))) return MGEMM_ERR_INVALID_ARG;
    if (!fits(M, N, K)) return MGEMM_ERR_UNSUPPORTED;
    const Plan p = make_plan(layoutW, M, N, K, X, ldx, Wg, Wu, ldw, false, again, dX != nullptr, dWg != nullptr);
    char* w;
    if (const mgemm_status_t st = check_work(p, work, work_bytes, &w); st != MGEMM_SUCCESS) return st;
    // Extents of dG and dU that the products see: padded with zeros where the
    // operand they meet is.
    const int64_t Mp = p.copy_x ? p.d_rows : M, Np = p.copy_w ? p.d_cols : N, ldd = p.d_cols;
    BlockArgs fa = base_args(h->ws, Mp, Np, p.copy_x && p.copy_w ? up(K, SLICE) : K), xa = base_args(h->ws, M, K, Np),
              wa = col ? base_args(h->ws, N, K, Mp) : base_args(h->ws, K, N, Mp);
    (col ? wa.batches_m : wa.batches_n) = 2;
    Grid fg{}, xg{}, wg{};
    Grids xs, ws;
    if (again) fg = fastest(grids_of(h, mgemm::BLOCK_AGAIN, fa));
    if (dX) xg = fastest(xs = grids_of(h, mgemm::BLOCK_DX, xa));
    if (dWg) wg = fastest(ws = grids_of(h, mgemm::BLOCK_DW, wa));
    if ((again && fg.wgs == 0) || (dX && xg.wgs == 0) || (dWg && wg.wgs == 0)) return MGEMM_ERR_UNSUPPORTED;
    const bool pair = dX && dWg && choose_pair(h, xs, ws, xg, wg);
    Operands o{X, Wg, Wu, ldx, ldw};
    if (const mgemm_status_t st = lay_out(p, w, o, stream); st != MGEMM_SUCCESS) return st;
    void *dG = w + p.dg_at, *dU = w + p.du_at;

    hipError_t e;
    if (again) {
        fa.A[0] = fa.A[1] = o.X; fa.lda = o.ldx;
        fa.B[0] = o.Wg; fa.B[1] = o.Wu; fa.ldb = o.ldw;
        fa.dZ = dZ; fa.ldz = lddz;
        fa.Mz = M; fa.Nz = N;
        fa.C[0] = dG; fa.C[1] = dU; fa.ldc = ldd;
        e = mgemm::launch_block_forward(fa, (int)dtype, col, true, fg.tile, stream);
    } else {
        e = mgemm::launch_gated_grad(M, N, p.d_rows, p.d_cols, G, U, ldg, dZ, lddz, dG, dU, ldd, (int)dtype, stream);
    }
    if (e != hipSuccess) return MGEMM_ERR_HIP;
    const void* d[2] = {dG, dU};
    for (int i = 0; i < 2; ++i) {
        xa.A[i] = d[i];
        xa.B[i] = i ? o.Wu : o.Wg;
        xa.C[i] = dX;
        wa.A[i] = col ? d[i] : o.X;
        wa.B[i] = col ? o.X : d[i];
        wa.C[i] = i ? dWu : dWg;
    }
    xa.lda = ldd;
    xa.ldb = o.ldw;
    xa.ldc = lddx;
    wa.lda = col ? ldd : o.ldx;
    wa.ldb = col ? o.ldx : ldd;
    wa.ldc = lddw;
    wa.beta = beta;
    // Row-major weights (in x out) are contiguous along dX's contraction.
    if (pair) return status(mgemm::launch_block_pair(xa, wa, (int)dtype, !col, xg.tile.ks, wg.tile.ks, stream));
    if (dX) e = mgemm::launch_block_dx(xa, (int)dtype, !col, xg.tile, stream);
    if (dWg && e == hipSuccess) e = mgemm::launch_block_dw(wa, (int)dtype, wg.tile, stream);
    return status(e);
}

}  // extern "C"
