// Tile loop of the gated block's products (k_gated_forward.hip, k_gated_dx.hip,
// k_gated_dw.hip): 16-bit operands copied straight into a four-slot LDS ring
// of 32-element slices, fragments read one K-step ahead of the MFMAs that use
// them, one workgroup barrier per slice, and the order of copies, reads and
// MFMAs pinned so that one wave per SIMD keeps its matrix core fed: the
// schedule and LDS layouts of k_h_dma.hip.  What differs is how operands are
// found:
//   forward  one A (X) against the two weights in one tile, 96 columns of
//            each, so that a lane holds G and U of the same outputs and X is
//            read once;
//   dX       the contraction runs over two segments (dG with Wg, then dU with
//            Wu) into one accumulator: no second pass over dX, one rounding;
//   dW       both gradients in one grid: a tile's batch picks its matrices.
// A segment or batch changes base addresses only, by an offset that is the
// same for every lane, so the loop is one and the same.
//
// Split contraction: FP32 partial sums of whole-slice ranges, added in range
// order by a second launch (no atomics: results do not depend on timing).
#pragma once
#include "gated.h"

namespace mgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int BK = 32, NT = 256;
constexpr int SLOTS = 4, AHEAD = SLOTS - 1;      // slices in flight
constexpr int ROW = BK * 2;                      // bytes of a K-contiguous row of a slice
constexpr int SPLIT_GROUP_M = 2, UNSPLIT_GROUP_M = 4;   // tile orders of k_h_dma.hip

template <int FORM>
constexpr bool is_dual() { return FORM == BLOCK_FORWARD || FORM == BLOCK_AGAIN; }

// Plain forms: waves 2x2.  Forward: waves 4x1, a wave holds all 192 columns.
template <int FORM, int BM_, int BN_>
struct Cfg {
    static constexpr bool DUAL = is_dual<FORM>();
    static constexpr int BM = BM_, BN = BN_;
    static_assert(BN == 256 || BN == 192, "tile width");
    static_assert(!DUAL || BN == 192, "the forward pair uses the 192-wide slot");
    static_assert(BM == 256 || BM == 128, "tile height");
    static constexpr int A_BYTES = BM * ROW, A_COPIES = BM / 64;     // 1 KiB copies per wave per slice
    static constexpr int B_ROW = BN * 2, B_CHUNKS = BN / 8;
    static constexpr int B_BYTES = BK * B_ROW, B_COPIES = BN / 64;
    static constexpr int COPIES = A_COPIES + B_COPIES;
    static constexpr int SLOT_BYTES = A_BYTES + B_BYTES, LDS = SLOTS * SLOT_BYTES;
    static constexpr int WROWS = DUAL ? BM / 4 : BM / 2;
    static constexpr int TM = WROWS / 32, TN = DUAL ? BN / 32 : BN / 64;
    static constexpr int WN = DUAL ? 0 : BN / 2;
    static constexpr int OUT = DUAL ? BN / 2 : BN;
};

__device__ __forceinline__ int row_swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }
// Chunk position of chunk c in K-row k of a slot whose K-rows are W elements
// wide (an involution for each k): free of bank conflicts for the transposed reads.
template <int W>
__device__ __forceinline__ int chunk_pos(int c, int k) {
    if constexpr (W == 192) return (c & ~7) | ((c & 7) ^ (int)((0x6204035651271642ull >> ((k & 15) * 4)) & 7));
    else return c ^ ((0xCA60 >> ((k & 3) * 4)) & 15);
}

template <int DT>
__device__ __forceinline__ f32x16 mfma(i32x4 a, i32x4 b, f32x16 c) {
    if constexpr (DT == F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b),
                                                       c, 0, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
// Waits until at most n slices of L copies each are in flight (copies complete in order).
template <int L>
__device__ __forceinline__ void wait_slices(int n) {
    if (n <= 0) wait_vm<0>();
    else if (n == 1) wait_vm<L>();
    else wait_vm<2 * L>();
}
__device__ __forceinline__ void fence_sched() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}
__device__ __forceinline__ void slice_barrier() {
    fence_sched();
    __builtin_amdgcn_s_barrier();
    fence_sched();
}

template <int TM, int TN>
struct Frags {
    i32x4 a[TM];
    i32x4 b[TN];
};

// s = 1 / (1 + e^-g) from the hardware exp2 and reciprocal (relative errors
// near 1e-6, far below the 16-bit roundings that follow); e^g where 1 + e^-g
// would round to e^-g, so that e^-g does not overflow.
__device__ __forceinline__ float sigmoid_f32(float g) {
    constexpr float LOG2E = 1.44269504088896341f;
    const bool tail = !(g >= -20.0f);            // also NaN in, NaN out
    const float e = __builtin_amdgcn_exp2f(tail ? g * LOG2E : -g * LOG2E);
    return tail ? e : __builtin_amdgcn_rcpf(1.0f + e);
}
__device__ __forceinline__ void gated_grad(float g, float u, float dz, float& dg, float& du) {
    const float s = sigmoid_f32(g);
    du = dz * (g * s);
    dg = dz * u * (s * fmaf(g, 1.0f - s, 1.0f));
    // Both products are rounded to FP32 here.  Left to itself the compiler
    // folds some of them into the conversion to FP16 that follows (one
    // rounding in place of two), in one caller and not in another, and
    // recomputed G and U would not give the bits of stored ones.
    asm("" : "+v"(dg), "+v"(du));
}

// Four consecutive 16-bit elements of a row (zero past lim).
template <int DT>
__device__ __forceinline__ void load4(const uint16_t* row, int n, int lim, bool vec_ok, float (&v)[4]) {
    if (vec_ok && n + 4 <= lim) {
        const uint2 w = *(const uint2*)(row + n);
        v[0] = from_bits<DT>((uint16_t)w.x);
        v[1] = from_bits<DT>((uint16_t)(w.x >> 16));
        v[2] = from_bits<DT>((uint16_t)w.y);
        v[3] = from_bits<DT>((uint16_t)(w.y >> 16));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = n + e < lim ? from_bits<DT>(row[n + e]) : 0.0f;
    }
}
__device__ __forceinline__ bool vec4_ok(const void* p, int64_t ld) { return ld % 4 == 0 && ((uintptr_t)p & 7) == 0; }

// Stores the outputs of columns n0+ni .. n0+ni+3 of row m from their FP32
// sums: g alone (dX, dW) or g and u (forward).  Each output is rounded once;
// Z comes from the unrounded sums, dG and dU from G and U as the forward pass
// stores them.
template <int DT, int FORM>
__device__ __forceinline__ void block_out(const BlockArgs& f, int bt, int64_t m, int64_t n0, int ni, int nlim,
                                          f32x4 g, f32x4 u) {
    if (ni >= nlim) return;
    if constexpr (FORM == BLOCK_FORWARD) {
        float z[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = silu_f32<DT>(g[e]) * u[e];
        store_out4<DT, EPI_NONE>((uint16_t*)f.Z + m * f.ldz + n0, ni, nlim, vec4_ok(f.Z, f.ldz), 0.f, z);
        if (f.C[0] != nullptr) {
            float a[4] = {g[0], g[1], g[2], g[3]}, b[4] = {u[0], u[1], u[2], u[3]};
            store_out4<DT, EPI_NONE>((uint16_t*)f.C[0] + m * f.ldc + n0, ni, nlim, vec4_ok(f.C[0], f.ldc), 0.f, a);
            store_out4<DT, EPI_NONE>((uint16_t*)f.C[1] + m * f.ldc + n0, ni, nlim, vec4_ok(f.C[1], f.ldc), 0.f, b);
        }
    } else if constexpr (FORM == BLOCK_AGAIN) {
        float dz[4], a[4], b[4];
        load4<DT>((const uint16_t*)f.dZ + m * f.ldz + n0, ni, nlim, vec4_ok(f.dZ, f.ldz), dz);
#pragma unroll
        for (int e = 0; e < 4; ++e) gated_grad(round_trip<DT>(g[e]), round_trip<DT>(u[e]), dz[e], a[e], b[e]);
        store_out4<DT, EPI_NONE>((uint16_t*)f.C[0] + m * f.ldc + n0, ni, nlim, vec4_ok(f.C[0], f.ldc), 0.f, a);
        store_out4<DT, EPI_NONE>((uint16_t*)f.C[1] + m * f.ldc + n0, ni, nlim, vec4_ok(f.C[1], f.ldc), 0.f, b);
    } else {
        float v[4] = {g[0], g[1], g[2], g[3]};
        store_out4<DT, EPI_NONE>((uint16_t*)f.C[bt] + m * f.ldc + n0, ni, nlim, vec4_ok(f.C[bt], f.ldc), f.beta, v);
    }
}

template <int DT, int FORM, int BM, int BN, bool AMC, bool BKC, bool PARTIAL>
__global__ __launch_bounds__(NT, 1) void k_block(BlockArgs f) {
    using G = Cfg<FORM, BM, BN>;
    constexpr bool DUAL = G::DUAL;
    constexpr int SEGS = FORM == BLOCK_DX ? 2 : 1;
    static_assert(!(AMC && (BKC || DUAL)), "operand forms");
    constexpr int TM = G::TM, TN = G::TN, COPIES = G::COPIES, A_COPIES = G::A_COPIES;
    constexpr int A_BYTES = G::A_BYTES, A_KROW = BM * 2, A_CHUNKS = BM / 8, B_ROW = G::B_ROW;
    using Fr = Frags<TM, TN>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = DUAL ? wave : wave >> 1, wn = DUAL ? 0 : wave & 1;
    const int tiles_m = (int)((f.M + BM - 1) / BM), tiles_n = (int)((f.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(blockIdx.x, gridDim.x);
    const int split = pos % f.ksplit;
    int tmi, tni;
    tile_from_linear(pos / f.ksplit, tiles_m * f.batches_m, tiles_n * f.batches_n,
                     f.ksplit > 1 ? SPLIT_GROUP_M : UNSPLIT_GROUP_M, tmi, tni);
    const int tile = tmi * (tiles_n * f.batches_n) + tni;
    const int bt = tmi >= tiles_m || tni >= tiles_n;
    if (tmi >= tiles_m) tmi -= tiles_m;
    if (tni >= tiles_n) tni -= tiles_n;
    const int64_t m0 = (int64_t)tmi * BM, n0 = (int64_t)tni * G::OUT;
    const int mlim = (int)(f.M - m0 < BM ? f.M - m0 : BM);
    const int nlim = (int)(f.N - n0 < G::OUT ? f.N - n0 : G::OUT);
    const int nk_seg = (int)(f.K / BK), nk_all = SEGS * nk_seg;      // whole slices
    const int j0 = split * f.nks;                                    // this range's first slice
    const int nk = nk_all - j0 < f.nks ? nk_all - j0 : f.nks;
    const char* A = (const char*)f.A[FORM == BLOCK_DW ? bt : 0];
    const char* B = (const char*)f.B[FORM == BLOCK_DW ? bt : 0];
    // From the first half's matrices to the second's: dX's segments, the forward pair's second weight.
    const int64_t a_diff = (const char*)f.A[1] - (const char*)f.A[0];
    const int64_t b_diff = (const char*)f.B[1] - (const char*)f.B[0];

    // Copies of this wave, 1 KiB each (16 bytes a lane).  K-contiguous
    // operands: 16 rows of 64 bytes, lane l takes row l/4's chunk (l%4 ^ swz);
    // the others: 64 consecutive chunk positions of the slot.  Rows and
    // chunks past the edge read the last valid ones.
    const char* src[COPIES];
    int dst[COPIES];
#pragma unroll
    for (int i = 0; i < A_COPIES; ++i) {
        if constexpr (AMC) {
            const int j = wave * A_COPIES + i, q = 64 * j + lane, k = q / A_CHUNKS;
            int c = chunk_pos<BM>(q % A_CHUNKS, k);
            const int64_t left = (f.Mr - m0) / 8 - 1;
            c = c <= left ? c : (int)left;
            src[i] = A + ((int64_t)k * f.lda + m0 + 8 * c) * 2;
            dst[i] = j * 1024;
        } else {
            const int r0 = BM / 4 * wave + 16 * i, r = r0 + (lane >> 2);
            const int c = (lane & 3) ^ row_swz(r);
            src[i] = A + ((m0 + (r < mlim ? r : mlim - 1)) * f.lda + 8 * c) * 2;
            dst[i] = r0 * ROW;
        }
    }
#pragma unroll
    for (int i = 0; i < G::B_COPIES; ++i) {
        if constexpr (BKC) {
            const int r0 = BN / 4 * wave + 16 * i, r = r0 + (lane >> 2);
            const int c = (lane & 3) ^ row_swz(r);
            const bool second = DUAL && r >= G::OUT;
            int rr = second ? r - G::OUT : r;
            rr = rr < nlim ? rr : nlim - 1;
            src[A_COPIES + i] = B + (second ? b_diff : 0) + ((n0 + rr) * f.ldb + 8 * c) * 2;
            dst[A_COPIES + i] = A_BYTES + r0 * ROW;
        } else {
            const int j = wave * G::B_COPIES + i, q = 64 * j + lane, k = q / G::B_CHUNKS;
            int c = chunk_pos<BN>(q % G::B_CHUNKS, k);
            const bool second = DUAL && c >= G::OUT / 8;
            if (second) c -= G::OUT / 8;
            const int64_t left = (f.Nr - n0) / 8 - 1;
            c = c <= left ? c : (int)left;
            src[A_COPIES + i] = B + (second ? b_diff : 0) + ((int64_t)k * f.ldb + n0 + 8 * c) * 2;
            dst[A_COPIES + i] = A_BYTES + j * 1024;
        }
    }
    const int64_t a_step = AMC ? (int64_t)BK * f.lda * 2 : ROW, b_step = BKC ? ROW : (int64_t)BK * f.ldb * 2;
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
    // Byte offsets of slice j (of the whole contraction) from src.
    auto a_at = [&](int j) { return SEGS == 2 && j >= nk_seg ? a_diff + (j - nk_seg) * a_step : j * a_step; };
    auto b_at = [&](int j) { return SEGS == 2 && j >= nk_seg ? b_diff + (j - nk_seg) * b_step : j * b_step; };
    auto copy = [&](int s, int i) {
        copy_to_lds(src[i] + (i < A_COPIES ? a_at(j0 + s) : b_at(j0 + s)),
                    lds0 + (unsigned)(s % SLOTS) * G::SLOT_BYTES + dst[i]);
    };

    // Fragment read offsets within a slot.
    int a_off[TM][2][AMC ? 2 : 1], b_off[TN][2][BKC ? 1 : 2];
    const int q4 = lane >> 4, t16 = lane & 15;
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if constexpr (AMC) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 16 + 8 * (q4 >> 1) + 4 * h + (t16 >> 2);
                    const int m = G::WROWS * wm + 32 * t + 16 * (q4 & 1) + 4 * (t16 & 3);
                    a_off[t][ks][h] = k * A_KROW + (chunk_pos<BM>(m >> 3, k) << 4) + ((m & 7) << 1);
                }
            } else {
                const int r = G::WROWS * wm + 32 * t + (lane & 31);
                a_off[t][ks][0] = r * ROW + (((2 * ks + (lane >> 5)) ^ row_swz(r)) << 4);
            }
        }
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if constexpr (BKC) {
                const int r = G::WN * wn + 32 * t + (lane & 31);
                b_off[t][ks][0] = A_BYTES + r * ROW + (((2 * ks + (lane >> 5)) ^ row_swz(r)) << 4);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 16 + 8 * (q4 >> 1) + 4 * h + (t16 >> 2);
                    const int n = G::WN * wn + 32 * t + 16 * (q4 & 1) + 4 * (t16 & 3);
                    b_off[t][ks][h] = A_BYTES + k * B_ROW + (chunk_pos<BN>(n >> 3, k) << 4) + ((n & 7) << 1);
                }
            }
        }
    auto read_tr = [&](const unsigned char* lo, const unsigned char* hi) {
        const int2 l = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                    (__attribute__((address_space(3))) i16x4*)lo));
        const int2 h = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                    (__attribute__((address_space(3))) i16x4*)hi));
        return i32x4{l.x, l.y, h.x, h.y};
    };
    // Read r of (slice s, K-step ks), in the order the next K-step needs them:
    // A0, B0 .. B(TN-1), A1 .. A(TM-1).
    auto read = [&](Fr& fr, int s, int ks, int r) {
        const unsigned char* base = smem + (s % SLOTS) * G::SLOT_BYTES;
        if (r == 0 || r > TN) {
            const int t = r == 0 ? 0 : r - TN;
            if constexpr (AMC) fr.a[t] = read_tr(base + a_off[t][ks][0], base + a_off[t][ks][AMC]);
            else fr.a[t] = *(const i32x4*)(base + a_off[t][ks][0]);
        } else {
            if constexpr (BKC) fr.b[r - 1] = *(const i32x4*)(base + b_off[r - 1][ks][0]);
            else fr.b[r - 1] = read_tr(base + b_off[r - 1][ks][0], base + b_off[r - 1][ks][!BKC]);
        }
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    // One K-step: the MFMAs on `use`, with the reads of (rs, rks) and the
    // copies c0 .. c1-1 of slice cs spread between them.
    constexpr int NM = TM * TN, NR = TM + TN;
    auto kstep = [&](const Fr& use, Fr& nxt, bool do_read, int rs, int rks, bool do_copy, int cs, int c0, int c1) {
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            const int tm = i / TN, tn = (tm & 1) ? TN - 1 - i % TN : i % TN;
            acc[tm][tn] = mfma<DT>(use.b[tn], use.a[tm], acc[tm][tn]);
            if (do_copy) {
#pragma unroll
                for (int c = c0; c < c1; ++c)
                    if (i == (c - c0) * NM / (c1 - c0)) copy(cs, c);
            }
            if (do_read) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if ((r + 1 < NM ? r + 1 : NM - 1) == i) read(nxt, rs, rks, r);
            }
            fence_sched();
        }
    };

    // Prologue: request slices 0 .. AHEAD-1, make slice 0 visible, read its first fragments.
    Fr f0, f1;
    const int npro = nk < AHEAD ? nk : AHEAD;
    for (int s = 0; s < npro; ++s)
        for (int i = 0; i < COPIES; ++i) copy(s, i);
    if (nk > 0) {
        wait_slices<COPIES>(npro - 1);
        slice_barrier();
#pragma unroll
        for (int r = 0; r < NR; ++r) read(f0, 0, 0, r);
    }
    // Slice j: wait for this wave's copies of slice j+1 (later ones may stay
    // in flight), barrier (slice j+1 visible, the slot of slice j-1 free),
    // then K-step 0 with the A copies of slice j+AHEAD and K-step 1 with its
    // B copies.
    int j = 0;
    for (; j + AHEAD < nk; ++j) {
        wait_slices<COPIES>(AHEAD - 2);
        slice_barrier();
        kstep(f0, f1, true, j, 1, true, j + AHEAD, 0, A_COPIES);
        kstep(f1, f0, true, j + 1, 0, true, j + AHEAD, A_COPIES, COPIES);
    }
    for (; j < nk; ++j) {
        const bool next = j + 1 < nk;
        if (next) {
            wait_slices<COPIES>(nk - j - 2);
            slice_barrier();
        }
        kstep(f0, f1, true, j, 1, false, 0, 0, 1);
        kstep(f1, f0, next, j + 1, 0, false, 0, 0, 1);
    }

    // Contraction tail: the range that ends at the last whole slice adds the
    // remaining K % 32 of every segment, staged by ordinary loads into the
    // positions that the copies fill, zeros past K in both operands (only
    // k < K is read).  No copy is in flight any more.
    const int ktail = (int)(f.K - (int64_t)nk_seg * BK);
    if (ktail > 0 && j0 + nk == nk_all) {
#pragma unroll 1
        for (int seg = 0; seg < SEGS; ++seg) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < COPIES; ++i) {
                const bool is_a = i < A_COPIES;
                const int ib = i - A_COPIES;
                const uint16_t* s = (const uint16_t*)(src[i] + (is_a ? nk_seg * a_step + (seg ? a_diff : 0)
                                                                     : nk_seg * b_step + (seg ? b_diff : 0)));
                const bool k_runs = is_a ? !AMC : BKC;
                i32x4 v = i32x4{0, 0, 0, 0};
                if (!k_runs) {
                    const int k = is_a ? (64 * (wave * A_COPIES + i) + lane) / A_CHUNKS
                                       : (64 * (wave * G::B_COPIES + ib) + lane) / G::B_CHUNKS;
                    if (k < ktail) v = *(const i32x4*)s;
                } else {
                    const int r = is_a ? BM / 4 * wave + 16 * i + (lane >> 2) : BN / 4 * wave + 16 * ib + (lane >> 2);
                    const int k = 8 * ((lane & 3) ^ row_swz(r));
                    if (k + 8 <= ktail) {
                        v = *(const i32x4*)s;
                    } else if (k < ktail) {
                        uint16_t e[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q) e[q] = k + q < ktail ? s[q] : (uint16_t)0;
                        v = __builtin_bit_cast(i32x4, e);
                    }
                }
                *(i32x4*)(smem + dst[i] + 16 * lane) = v;
            }
            __syncthreads();
#pragma unroll
            for (int r = 0; r < NR; ++r) read(f0, 0, 0, r);
            kstep(f0, f1, true, 0, 1, false, 0, 0, 1);
            kstep(f1, f0, false, 0, 0, false, 0, 0, 1);
        }
    }

    // Lane holds C(m, n..n+3), m = row within the 32x32 block.
    if constexpr (PARTIAL) {
        float* d = f.part + ((int64_t)tile * f.ksplit + split) * (int64_t)(NT * TM * TN * 16) + 4 * tid;
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            if (G::WROWS * wm + 32 * tm + (lane & 31) >= mlim) continue;
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& a = acc[tm][tn];
                    *(f32x4*)(d + (int64_t)((tm * TN + tn) * 4 + q) * NT * 4) =
                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
        }
    } else {
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            const int mi = G::WROWS * wm + 32 * tm + (lane & 31);
            if (mi >= mlim) continue;
#pragma unroll
            for (int tn = 0; tn < (DUAL ? TN / 2 : TN); ++tn)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& a = acc[tm][tn];
                    const f32x16& b = acc[tm][DUAL ? tn + TN / 2 : tn];
                    block_out<DT, FORM>(f, bt, m0 + mi, n0, G::WN * wn + 32 * tn + 8 * q + 4 * (lane >> 5), nlim,
                                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]},
                                        f32x4{b[4 * q], b[4 * q + 1], b[4 * q + 2], b[4 * q + 3]});
                }
        }
    }
}

// Second phase of a split: one thread per 16-byte chunk of a tile's
// accumulators sums the ranges in range order and stores four outputs.
template <int DT, int FORM, int BM, int BN>
__global__ __launch_bounds__(NT) void k_block_reduce(BlockArgs f) {
    using G = Cfg<FORM, BM, BN>;
    constexpr bool DUAL = G::DUAL;
    constexpr int TM = G::TM, TN = G::TN, TNO = DUAL ? TN / 2 : TN, CH = TM * TNO * 4;
    constexpr int64_t TILE = (int64_t)NT * TM * TN * 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = DUAL ? wave : wave >> 1, wn = DUAL ? 0 : wave & 1;
    const int tiles_m = (int)((f.M + BM - 1) / BM), tiles_n = (int)((f.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(blockIdx.x, gridDim.x);
    const int c = pos % CH;
    int tmi, tni;
    tile_from_linear(pos / CH, tiles_m * f.batches_m, tiles_n * f.batches_n, SPLIT_GROUP_M, tmi, tni);
    const int tile = tmi * (tiles_n * f.batches_n) + tni;
    const int bt = tmi >= tiles_m || tni >= tiles_n;
    if (tmi >= tiles_m) tmi -= tiles_m;
    if (tni >= tiles_n) tni -= tiles_n;
    const int tm = c / (TNO * 4), tn = (c / 4) % TNO, q = c % 4;
    const int64_t m0 = (int64_t)tmi * BM, n0 = (int64_t)tni * G::OUT;
    const int nlim = (int)(f.N - n0 < G::OUT ? f.N - n0 : G::OUT);
    const int64_t m = m0 + G::WROWS * wm + 32 * tm + (lane & 31);
    const int ni = G::WN * wn + 32 * tn + 8 * q + 4 * (lane >> 5);
    if (m >= f.M || ni >= nlim) return;
    const float* part = f.part + (int64_t)tile * f.ksplit * TILE + 4 * tid;
    auto sum = [&](int chunk) {
        const float* p = part + (int64_t)chunk * NT * 4;
        f32x4 a = *(const f32x4*)p;
        int s = 1;
        for (; s + 4 <= f.ksplit; s += 4) {
            const f32x4 b0 = *(const f32x4*)(p + s * TILE), b1 = *(const f32x4*)(p + (s + 1) * TILE);
            const f32x4 b2 = *(const f32x4*)(p + (s + 2) * TILE), b3 = *(const f32x4*)(p + (s + 3) * TILE);
            a = (((a + b0) + b1) + b2) + b3;
        }
        for (; s < f.ksplit; ++s) a = a + *(const f32x4*)(p + s * TILE);
        return a;
    };
    const f32x4 g = sum((tm * TN + tn) * 4 + q);
    if constexpr (DUAL) block_out<DT, FORM>(f, bt, m, n0, ni, nlim, g, sum((tm * TN + tn + TN / 2) * 4 + q));
    else block_out<DT, FORM>(f, bt, m, n0, ni, nlim, g, g);
}

template <int DT, int FORM, int BM, int BN, bool AMC, bool BKC>
hipError_t launch_block(BlockArgs a, int ks, hipStream_t s) {
    using G = Cfg<FORM, BM, BN>;
    const int64_t slices = (a.K / BK) * (FORM == BLOCK_DX ? 2 : 1);
    a.nks = (int)(ks > 1 ? (slices + ks - 1) / ks : (slices > 0 ? slices : 1));
    a.ksplit = ks > 1 ? (int)((slices + a.nks - 1) / a.nks) : 1;
    const int64_t tiles = ((a.M + BM - 1) / BM) * a.batches_m * (((a.N + G::OUT - 1) / G::OUT) * a.batches_n);
    auto go = [&](auto kern, bool (&done)[MAX_DEVICES]) -> hipError_t {
        if (hipError_t e = set_lds_limit_once((const void*)kern, G::LDS, done); e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * a.ksplit)), dim3(NT), G::LDS, s, a);
        return hipGetLastError();
    };
    if (a.ksplit == 1) {
        static bool done[MAX_DEVICES] = {};
        return go(k_block<DT, FORM, BM, BN, AMC, BKC, false>, done);
    }
    static bool done[MAX_DEVICES] = {};
    if (hipError_t e = go(k_block<DT, FORM, BM, BN, AMC, BKC, true>, done); e != hipSuccess) return e;
    constexpr int CH = G::TM * (G::DUAL ? G::TN / 2 : G::TN) * 4;
    hipLaunchKernelGGL((k_block_reduce<DT, FORM, BM, BN>), dim3((unsigned)(tiles * CH)), dim3(NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace mgemm
