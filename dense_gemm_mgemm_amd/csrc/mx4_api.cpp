// Entry points of the microscaled 4-bit format: argument checks, kernel
// choice, and the workspace of activations quantised within a call.  See
// include/mgemm.h for the contracts.
#include <hip/hip_runtime.h>

#include "host.h"
#include "mx4.h"

using namespace mgemm_host;

namespace {

using mgemm::Mx4Args;
using mgemm::Workspace;

constexpr int64_t LIM = (int64_t)1 << 62;

bool valid_dtype(mgemm_dtype_t d) { return d == MGEMM_F32 || d == MGEMM_F16 || d == MGEMM_BF16; }
int64_t max1(int64_t x) { return x > 1 ? x : 1; }
mgemm_status_t status(hipError_t e) { return e == hipSuccess ? MGEMM_SUCCESS : MGEMM_ERR_HIP; }

// Whether rows x K values with element stride ld can be addressed.
bool valid_matrix(int64_t rows, int64_t K, int64_t ld) {
    return ld >= max1(K) && (rows == 0 || ld <= LIM / rows);
}
// The same for a matrix of codes and scales with byte strides.
bool valid_mx4(int64_t rows, int64_t K, int64_t ldq, int64_t lds) {
    if (K > LIM / 2) return false;
    const int64_t nb = mgemm::mx4_blocks(K);
    return ldq >= max1(16 * nb) && lds >= max1(nb) && (rows == 0 || (ldq <= LIM / rows && lds <= LIM / rows));
}

// What mgemm_run_mx4 and mgemm_set_mx4_kernel accept.
bool valid_kernel(mgemm_kernel_t kernel, int32_t ksplit) {
    if (ksplit < 0 || ksplit > MGEMM_MAX_KSPLIT) return false;
    if (kernel == MGEMM_KERNEL_AUTO) return ksplit == 0;
    return kernel >= MGEMM_KERNEL_MX4_GENERAL && kernel <= MGEMM_KERNEL_MX4_MFMA_64;
}

Problem problem(mgemm_handle_t h, int64_t M, int64_t N, int64_t K, void* C, int64_t ldc, mgemm_dtype_t ctype) {
    Problem p{};
    p.M = M; p.N = N; p.K = K;
    p.alpha = 1.0f;
    p.a_kc = p.b_kc = 1;
    p.C = C; p.ldc = ldc;
    p.dtype = (int)ctype;
    p.num_cu = h->num_cu;
    p.epilogue = mgemm::EPI_NONE;
    p.stamps = h->stamps;
    p.stamps_cap = h->stamps ? h->stamps_cap : 0;
    return p;
}

struct Tile {
    int bn, bm, ks;
};
struct Shape {
    mgemm_kernel_t kernel;
    int bn, bm;
};
constexpr Shape SHAPES[] = {{MGEMM_KERNEL_MX4_MFMA, 256, 256},
                            {MGEMM_KERNEL_MX4_MFMA_192, 192, 256},
                            {MGEMM_KERNEL_MX4_MFMA_128, 192, 128},
                            {MGEMM_KERNEL_MX4_MFMA_64, 192, 64}};

// A tile's rate in the time model, from what a 128-element slice of it takes:
// 64x192 0.5 us, 128x192 0.75 (0.58 for few rows, which stream the weights from
// HBM whatever they compute), 256x192 1.0, 256x256 1.22.  Medians on three cards,
// codes given: 300 x 5000 x 2000 on 64 / 128 rows 12.3 to 12.7 / 16.6 to 16.9 us;
// 1000^3 8.3 to 8.8 / 11.1 to 11.4; 8192 x 12288 x 4096 on 64 / 128 / 256 x 192 and 256 x
// 256 442 to 456 / 410 / 326 / 303; 48 x 12288 x 4096 whole 18.6, in 4 ranges 12.4 to
// 13.6.  These are a few shapes, laid over a model of 16-bit products: it prices
// the gated pair's splits too high (32 and 64 rows x 12288 x 4096 run whole in 30
// us; in two ranges they take 22.6 and 24.6).
double tile_speed(const Problem& p, int bn, int bm) {
    if (bm == 64) return 0.37;
    if (bm == 128) return p.M <= 128 ? 0.63 : 0.49;
    return bn == 256 ? 0.80 : 0.735;
}

// The split with the smallest predicted time for one tile shape.  A
// 128-element slice moves the bytes and takes the matrix time of a 32-element
// slice of a 16-bit product, so the 16-bit time model applies to K / 4, with the
// partials priced as for FP8.
Tile best_split(const Problem& p, int bn, int bm, const Workspace& ws, double* t_out) {
    Problem q = p;
    q.K = p.K / 4;
    const int out = p.B2 != nullptr ? 96 : bn;
    Tile best{bn, bm, 1};
    double bt = 1e300;
    for (int req = 1, last = 0; req <= MGEMM_MAX_KSPLIT; ++req) {
        const int ks = mgemm::mx4_splits(p, bn, bm, req, ws);
        if (ks <= last) continue;
        last = ks;
        // (A range also costs the thread that adds it 0.3 us.)
        const double t = predict_us(q, bm, bn, out, tile_speed(p, bn, bm), 1, ks, 4.5e6) + (ks > 1 ? 0.3 * ks : 0.0);
        if (t < bt) { bt = t; best.ks = ks; }
    }
    *t_out = bt;
    return best;
}

// Predicted time (microseconds) of the decode kernel on codes: a launch, then
// per 4096 columns (a 16-column workgroup on each CU; the gated pair has both
// matrices') and 1024 elements of K (a slice for each wave) 0.023 us a row.
// Medians on three cards, 4096 x 12288 weights: M = 17 / 32 / 48 / 64 12.2 to 12.5 /
// 14.5 to 14.7 / 20.6 to 20.9 / 22.7 to 23.0 us, against 12.1 to 13.1 / 12.5 to 13.6 /
// 13.3 to 14.3 / 14.3 to 15.1 on 64-row tiles in 8 ranges; 12288 x 4096: M = 1 / 16 8.7 to
// 8.9 / 10.6 to 10.9 against 9.9 to 11.2 / 10.3 to 13.4 in 4; 40 x 1000 x 1000 6.0 to 9.3
// against 7.9 to 9.9 (the host bounds the shortest).
double skinny_us(const Problem& p) {
    const int64_t n = p.B2 != nullptr ? 2 * p.N : p.N;
    return 4.5 + (double)((n + 4095) / 4096) * (double)((p.K + 1023) / 1024) * 0.023 * (double)p.M;
}
// Launches a product of codes: forced kernel or the library's choice.
mgemm_status_t launch(const Problem& p, const Mx4Args& a, mgemm_kernel_t kernel, int ksplit, const Workspace& ws,
                      hipStream_t s) {
    if (kernel == MGEMM_KERNEL_MX4_GENERAL || kernel == MGEMM_KERNEL_MX4_SKINNY) {
        if (ksplit > 1) return MGEMM_ERR_UNSUPPORTED;
        if (kernel == MGEMM_KERNEL_MX4_GENERAL) return status(mgemm::launch_mx4_general(p, a, s));
        if (!mgemm::mx4_skinny_supports(p, a)) return MGEMM_ERR_UNSUPPORTED;
        return status(mgemm::launch_mx4_skinny(p, a, s));
    }
    Tile best{0, 0, 0};
    double best_t = 1e300;
    for (const Shape& c : SHAPES) {
        if (kernel != MGEMM_KERNEL_AUTO && kernel != c.kernel) continue;
        if (!mgemm::mx4_mfma_supports(p, a, c.bn, c.bm)) continue;
        double t;
        const Tile tile = best_split(p, c.bn, c.bm, ws, &t);
        if (t < best_t) { best_t = t; best = tile; }
    }
    if (kernel == MGEMM_KERNEL_AUTO) {
        if (mgemm::mx4_skinny_supports(p, a) && skinny_us(p) < best_t)
            return status(mgemm::launch_mx4_skinny(p, a, s));
        if (best.bn == 0) return status(mgemm::launch_mx4_general(p, a, s));
    }
    if (best.bn == 0) return MGEMM_ERR_UNSUPPORTED;
    if (ksplit > 0) best.ks = mgemm::mx4_splits(p, best.bn, best.bm, ksplit, ws);
    if (best.ks < 1) return MGEMM_ERR_UNSUPPORTED;
    return status(mgemm::launch_mx4_mfma(p, a, best.bn, best.bm, best.ks, ws, s));
}

// Y (or Z: p.B2 set) from activations: quantised inside the decode kernel, or
// into the workspace a band of rows at a time.
mgemm_status_t from_values(mgemm_handle_t h, Problem p, Mx4Args a, hipStream_t s) {
    const int es = a.xtype == mgemm::F32 ? 4 : 2, cs = p.dtype == mgemm::F32 ? 4 : 2;
    // The decode kernel's own quantisation is repeated by every workgroup and
    // grows with the rows it has room for (4 or 16) times K: 1.6 us at 16384
    // values (M = 1 .. 4, K = 4096: 10.6 to 10.8 us, from codes 8.7 to 9.5) and 7.6
    // at 65536; a launch of its own adds 2.2 (M = 8: 11.6 to 12.4 us).
    constexpr int64_t IN_KERNEL = 20480;
    const bool forced = h->mx4_kernel != MGEMM_KERNEL_AUTO;
    if (!forced && (p.M <= 4 ? 4 : 16) * p.K <= IN_KERNEL && mgemm::mx4_skinny_supports(p, a))
        return status(mgemm::launch_mx4_skinny(p, a, s));
    // Codes and scales take the front half of the workspace, split-K partials the rest.
    const int64_t nb = mgemm::mx4_blocks(p.K), ldq = 16 * nb, lds = (nb + 15) / 16 * 16;
    const int64_t half = h->ws.part_bytes / 2;
    int64_t band = half / (ldq + lds);
    if (band < 1) return MGEMM_ERR_UNSUPPORTED;
    if (band > 256) band = band / 256 * 256;
    Workspace rest = h->ws;
    rest.part = (char*)h->ws.part + half;
    rest.part_bytes -= half;
    const char* X = (const char*)a.X;
    char* C = (char*)p.C;
    const int64_t M = p.M;
    uint8_t* q = (uint8_t*)h->ws.part;
    a.X = nullptr;
    p.A = q;
    p.lda = ldq;
    a.ldsa = lds;
    for (int64_t m = 0; m < M; m += band) {
        p.M = M - m < band ? M - m : band;
        uint8_t* sc = q + p.M * ldq;
        a.sa = sc;
        p.C = C + m * p.ldc * cs;
        hipError_t e = mgemm::launch_quantize_mx4(p.M, p.K, X + m * a.ldx * es, a.ldx, a.xtype, q, ldq, sc, lds, s);
        if (e != hipSuccess) return MGEMM_ERR_HIP;
        const mgemm_status_t st = launch(p, a, h->mx4_kernel, h->mx4_ksplit, rest, s);
        if (st != MGEMM_SUCCESS) return st;
    }
    return MGEMM_SUCCESS;
}

}  // namespace

extern "C" {

mgemm_status_t mgemm_quantize_mx4(mgemm_handle_t h, int64_t M, int64_t K, const void* X, int64_t ldx,
                                  mgemm_dtype_t xtype, void* Q, int64_t ldq, void* S, int64_t lds,
                                  hipStream_t stream) {
    if (!h || M < 0 || K < 0 || !valid_dtype(xtype)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_matrix(M, K, ldx) || !valid_mx4(M, K, ldq, lds)) return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return MGEMM_SUCCESS;
    if (!X || !Q || !S) return MGEMM_ERR_INVALID_ARG;
    if (K > (int64_t)1 << 33) return MGEMM_ERR_UNSUPPORTED;
    return status(mgemm::launch_quantize_mx4(M, K, X, ldx, (int)xtype, (uint8_t*)Q, ldq, (uint8_t*)S, lds, stream));
}

mgemm_status_t mgemm_dequantize_mx4(mgemm_handle_t h, int64_t M, int64_t K, const void* Q, int64_t ldq,
                                    const void* S, int64_t lds, void* Y, int64_t ldy, mgemm_dtype_t ytype,
                                    hipStream_t stream) {
    if (!h || M < 0 || K < 0 || !valid_dtype(ytype)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_matrix(M, K, ldy) || !valid_mx4(M, K, ldq, lds)) return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || K == 0) return MGEMM_SUCCESS;
    if (!Q || !S || !Y) return MGEMM_ERR_INVALID_ARG;
    if (K > (int64_t)1 << 33) return MGEMM_ERR_UNSUPPORTED;
    return status(mgemm::launch_dequantize_mx4(M, K, (const uint8_t*)Q, ldq, (const uint8_t*)S, lds, Y, ldy,
                                               (int)ytype, stream));
}

mgemm_status_t mgemm_run_mx4(mgemm_handle_t h, mgemm_kernel_t kernel, int32_t ksplit, int64_t M, int64_t N,
                             int64_t K, float alpha, const void* A, int64_t lda, const void* SA, int64_t ldsa,
                             const void* B, int64_t ldb, const void* SB, int64_t ldsb, float beta, void* C,
                             int64_t ldc, mgemm_dtype_t ctype, hipStream_t stream) {
    if (!h || M < 0 || N < 0 || K < 0 || !valid_dtype(ctype)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_kernel(kernel, ksplit)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_mx4(M, K, lda, ldsa) || !valid_mx4(N, K, ldb, ldsb) || !valid_matrix(M, N, ldc))
        return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MGEMM_SUCCESS;
    if (!C) return MGEMM_ERR_INVALID_ARG;
    Problem p = problem(h, M, N, K, C, ldc, ctype);
    p.alpha = alpha;
    p.beta = beta;
    if (K == 0 || alpha == 0.f) return status(mgemm::launch_scale(p, stream));
    if (!A || !SA || !B || !SB) return MGEMM_ERR_INVALID_ARG;
    p.A = A; p.lda = lda;
    p.B = B; p.ldb = ldb;
    Mx4Args a{};
    a.sa = (const uint8_t*)SA; a.ldsa = ldsa;
    a.sb = (const uint8_t*)SB; a.ldsb = ldsb;
    return launch(p, a, kernel, ksplit, h->ws, stream);
}

mgemm_status_t mgemm_linear_mx4(mgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                                mgemm_dtype_t xtype, const void* B, int64_t ldb, const void* SB, int64_t ldsb,
                                void* Y, int64_t ldy, mgemm_dtype_t ytype, hipStream_t stream) {
    if (!h || M < 0 || N < 0 || K < 0 || !valid_dtype(xtype) || !valid_dtype(ytype)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_matrix(M, K, ldx) || !valid_mx4(N, K, ldb, ldsb) || !valid_matrix(M, N, ldy))
        return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MGEMM_SUCCESS;
    if (!Y) return MGEMM_ERR_INVALID_ARG;
    Problem p = problem(h, M, N, K, Y, ldy, ytype);
    if (K == 0) return status(mgemm::launch_scale(p, stream));
    if (!X || !B || !SB) return MGEMM_ERR_INVALID_ARG;
    p.B = B; p.ldb = ldb;
    Mx4Args a{};
    a.sb = (const uint8_t*)SB; a.ldsb = ldsb;
    a.X = X; a.ldx = ldx; a.xtype = (int)xtype;
    return from_values(h, p, a, stream);
}

mgemm_status_t mgemm_gated_mx4(mgemm_handle_t h, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                               mgemm_dtype_t xtype, const void* Bg, const void* SBg, const void* Bu,
                               const void* SBu, int64_t ldb, int64_t ldsb, void* Z, int64_t ldz,
                               mgemm_dtype_t ztype, hipStream_t stream) {
    if (!h || M < 0 || N < 0 || K < 0 || !valid_dtype(xtype) || !valid_dtype(ztype)) return MGEMM_ERR_INVALID_ARG;
    if (!valid_matrix(M, K, ldx) || !valid_mx4(N, K, ldb, ldsb) || !valid_matrix(M, N, ldz))
        return MGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return MGEMM_SUCCESS;
    if (!Z) return MGEMM_ERR_INVALID_ARG;
    Problem p = problem(h, M, N, K, Z, ldz, ztype);
    if (K == 0) return status(mgemm::launch_scale(p, stream));   // G = U = 0
    if (!X || !Bg || !SBg || !Bu || !SBu) return MGEMM_ERR_INVALID_ARG;
    p.B = Bg; p.B2 = Bu; p.ldb = p.ldb2 = ldb;
    Mx4Args a{};
    a.sb = (const uint8_t*)SBg; a.sb2 = (const uint8_t*)SBu; a.ldsb = ldsb;
    a.X = X; a.ldx = ldx; a.xtype = (int)xtype;
    return from_values(h, p, a, stream);
}

mgemm_status_t mgemm_set_mx4_kernel(mgemm_handle_t h, mgemm_kernel_t kernel, int32_t ksplit) {
    if (!h || !valid_kernel(kernel, ksplit)) return MGEMM_ERR_INVALID_ARG;
    h->mx4_kernel = kernel;
    h->mx4_ksplit = ksplit;
    return MGEMM_SUCCESS;
}

}  // extern "C"
