// Tile loop of the gated block's products (k_gated_forward.hip, k_gated_dx.hip,
// k_gated_dw.hip): 16-bit operands copied straight into an LDS ring of
// slices of 32 or 64 elements, fragments read ahead of the MFMAs that use them,
// one workgroup barrier per slice, and the order of copies, reads and
// MFMAs pinned so that one wave per SIMD keeps its matrix core fed: the
// schedule and LDS layouts of k_h_dma.hip.  What differs is how operands are
// found:
//   forward  one A (X) against the two weights in one tile, so that a lane
//            holds G and U of the same outputs and X is read once;
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

constexpr int NT = 256;
constexpr int SPLIT_GROUP_M = 2, UNSPLIT_GROUP_M = 4;   // tile orders of k_h_dma.hip
constexpr int LDS_MAX = 160 * 1024;

template <int FORM>
constexpr bool is_dual() { return FORM == BLOCK_FORWARD || FORM == BLOCK_AGAIN; }

// Square tiles, waves 2x2.  A forward tile's B slot holds T/2 columns of Wg,
// then the same T/2 of Wu; a wave takes the same columns of both, so that G
// and U of an output are in matching registers of one lane.
template <int FORM, int T>
struct Cfg {
    static constexpr bool DUAL = is_dual<FORM>();
    static constexpr int BM = T, BN = T;
    static_assert(T == 256 || T == 128, "tile size");
    // A slice of 64 is a 128-byte line of a K-contiguous row.  With 32 each
    // line is fetched twice, half of it used (128 x 128 tiles, both operands
    // K-contiguous: 0.31 us per 32 against 0.20); the 256 tile's ring has no
    // room for more than two slices of 64.
    static constexpr int BK = slice_of(BM), KS = BK / 16;            // elements and K-steps of a slice
    static constexpr int ROW = BK * 2;                               // bytes of a K-contiguous row of a slice
    static constexpr int A_BYTES = BM * ROW, A_COPIES = A_BYTES / 4096;   // 1 KiB copies per wave per slice
    static constexpr int B_ROW = BN * 2, B_CHUNKS = BN / 8;
    static constexpr int B_BYTES = BK * B_ROW, B_COPIES = B_BYTES / 4096;
    static constexpr int COPIES = A_COPIES + B_COPIES;
    static constexpr int SLOT_BYTES = A_BYTES + B_BYTES;
    // As many slices in flight as fit: all workgroups of an XCD walk the
    // contraction together, so each slice's first request goes to memory (1 to
    // 2 us under load).
    static constexpr int SLOTS = LDS_MAX / SLOT_BYTES, AHEAD = SLOTS - 1;
    static constexpr int WROWS = BM / 2, TM = WROWS / 32, TN = BN / 64;
    static constexpr int OUT = DUAL ? BN / 2 : BN;                   // output columns of a tile
    static constexpr int WOUT = OUT / 2;                             // of a wave
    static constexpr int TNO = DUAL ? TN / 2 : TN;                   // 32-column output blocks of a wave
    static constexpr int STAGE_ROW = WOUT * 2 + 16;                  // bytes of a staged row of outputs
    static constexpr int LDS = SLOTS * SLOT_BYTES;
    static_assert(4 * 3 * 32 * STAGE_ROW <= LDS, "outputs are staged in the ring");
    // Slot column of a wave's 32-column block t.
    static __device__ __forceinline__ int column(int wn, int t) {
        if constexpr (DUAL) return (t < TNO ? 0 : OUT) + WOUT * wn + 32 * (t % TNO);
        else return WOUT * wn + 32 * t;
    }
};

// Chunk c of a K-contiguous row r is at position c ^ row_swz(r): the 16-byte
// reads of a wave hit every bank once per 16 lanes.
template <int BK>
__device__ __forceinline__ int row_swz(int r) {
    if constexpr (BK == 64) return (r >> 1) & 7;
    else return ((r >> 1) ^ (r >> 2)) & 3;
}
// Chunk position of chunk c in K-row k of a slot whose K-rows are 128 or 256
// elements wide: free of bank conflicts for the transposed reads.
__device__ __forceinline__ int chunk_pos(int c, int k) { return c ^ ((0xCA60 >> ((k & 3) * 4)) & 15); }

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
// Waits until at most n <= MAX slices of L copies each are in flight (copies complete in order).
template <int L, int MAX>
__device__ __forceinline__ void wait_slices(int n) {
    if constexpr (MAX == 0) {
        wait_vm<0>();
    } else {
        if (n >= MAX) wait_vm<L * MAX>();
        else wait_slices<L, MAX - 1>(n);
    }
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

// Orders LDS accesses between the lanes of one wave: the hardware keeps a
// wave's LDS operations in order, so only the compiler has to be told.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A value into, and out of, an accumulator register at this point of the
// program.  Left to itself the compiler moves a whole tile's accumulators to
// vector registers before the first use, more than there are.
__device__ __forceinline__ float in_acc(float x) {
    asm volatile("" : "+a"(x));
    return x;
}
__device__ __forceinline__ float from_acc(float x) {
    float y;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(y) : "a"(x));
    return y;
}
// Before the first from_acc after MFMAs: longer than a matrix result takes to
// be readable (the compiler does not see into from_acc).
__device__ __forceinline__ void acc_settle() {
    fence_sched();
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    fence_sched();
}

template <int TM, int TN>
struct Frags {
    i32x4 a[TM];
    i32x4 b[TN];
};

// dG and dU of N outputs.  The sigmoid's power of two comes last (Gate): with a
// gate at -88 s is 6e-39, which FP32 arithmetic without subnormal exp2 results
// takes for 0, and dZ U s (1 + G) may still be any number.  Gates below -20 are
// rare, and their form costs nine more operations an output (dG and dU of 1024 x
// 12288: 4 us), so only waves that hold one take it; the other gives the same
// bits at -20 and above.
template <int N>
__device__ __forceinline__ void gated_grad(const float (&g)[N], const float (&u)[N], const float (&dz)[N],
                                           float (&dg)[N], float (&du)[N]) {
    bool far = false;
#pragma unroll
    for (int i = 0; i < N; ++i) far |= !(g[i] >= GATE_TAIL);
    if (far) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Gate s = gate_of(g[i]);
            const float rest = s.tail ? 1.0f : 1.0f - s.m;               // 1 - s
            du[i] = __builtin_amdgcn_ldexpf(dz[i] * (g[i] * s.m), s.e);
            dg[i] = __builtin_amdgcn_ldexpf(dz[i] * u[i] * (s.m * fmaf(g[i], rest, 1.0f)), s.e);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float s = near_sigmoid(g[i]);
            du[i] = dz[i] * (g[i] * s);
            dg[i] = dz[i] * u[i] * (s * fmaf(g[i], 1.0f - s, 1.0f));
        }
    }
    // Both products are rounded to FP32 here.  Left to itself the compiler
    // folds some of them into the conversion to FP16 that follows (one
    // rounding in place of two), in one caller and not in another, and
    // recomputed G and U would not give the bits of stored ones.
#pragma unroll
    for (int i = 0; i < N; ++i) asm("" : "+v"(dg[i]), "+v"(du[i]));
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

// Sums g and u of outputs (m, n .. n+3), rounded as the forward pass stores them,
// to dG and dU.  Past dZ, in the rows and columns that a copied operand is padded
// with, the results are zeros whatever the sums: 0 times an infinite weight is
// not.
template <int DT>
__device__ __forceinline__ void again_grad(const BlockArgs& f, int64_t m, int64_t n, f32x4& g, f32x4& u) {
    const int lim = m < f.Mz ? (int)(f.Nz - n < 4 ? f.Nz - n : 4) : 0;          // outputs that exist (none if <= 0)
    float gs[4], us[4], dz[4], a[4], b[4];
    load4<DT>((const uint16_t*)f.dZ + m * f.ldz + n, 0, lim, vec4_ok(f.dZ, f.ldz), dz);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        gs[e] = e < lim ? round_trip<DT>(g[e]) : 0.0f;
        us[e] = e < lim ? round_trip<DT>(u[e]) : 0.0f;
    }
    gated_grad(gs, us, dz, a, b);
    g = f32x4{a[0], a[1], a[2], a[3]};
    u = f32x4{b[0], b[1], b[2], b[3]};
}

// Four outputs of plane `plane` (forward: Z, G, U; recomputed backward: dG, dU)
// before their one rounding.  g: the sums of dX, dW or G, or dG; u: of U, or dU.
// Z comes from the unrounded sums.
template <int DT, int FORM, bool FAR>
__device__ __forceinline__ void block_value(int plane, f32x4 g, f32x4 u, float (&v)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (FORM == BLOCK_FORWARD)
            v[e] = plane == 0 ? gated_product<DT, FAR>(g[e], u[e]) : plane == 1 ? g[e] : u[e];
        else v[e] = plane == 0 ? g[e] : u[e];
    }
}
template <int FORM>
constexpr int planes() { return FORM == BLOCK_FORWARD ? 3 : FORM == BLOCK_AGAIN ? 2 : 1; }
// Plane's matrix (null: not stored) and its row stride.
template <int FORM>
__device__ __forceinline__ uint16_t* plane_of(const BlockArgs& f, int plane, int bt, int64_t& ld) {
    if constexpr (FORM == BLOCK_FORWARD) {
        ld = plane == 0 ? f.ldz : f.ldc;
        return (uint16_t*)(plane == 0 ? f.Z : plane == 1 ? f.C[0] : f.C[1]);
    } else {
        ld = f.ldc;
        return (uint16_t*)((FORM == BLOCK_AGAIN ? plane : bt) ? f.C[1] : f.C[0]);
    }
}

// What a workgroup stores: outputs, partial sums, or what f.ksplit says.
enum Store : int { STORE_OUT = 0, STORE_PART = 1, STORE_EITHER = 2 };

// Workgroup bid of nblocks.
template <int DT, int FORM, int T, bool AMC, bool BKC, int STORE>
__device__ __forceinline__ void block_body(const BlockArgs& f, int bid, int nblocks, unsigned char* smem) {
    using G = Cfg<FORM, T>;
    constexpr int BM = T, BN = T;
    constexpr bool DUAL = G::DUAL;
    constexpr int SEGS = FORM == BLOCK_DX ? 2 : 1;
    static_assert(!(AMC && (BKC || DUAL)), "operand forms");
    constexpr int TM = G::TM, TN = G::TN, COPIES = G::COPIES, A_COPIES = G::A_COPIES;
    constexpr int SLOTS = G::SLOTS, AHEAD = G::AHEAD, BK = G::BK, KS = G::KS, ROW = G::ROW;
    constexpr int RCH = ROW / 16, RPC = 64 / RCH;        // chunks of a K-contiguous row, and rows per copy
    constexpr int A_BYTES = G::A_BYTES, A_KROW = BM * 2, A_CHUNKS = BM / 8, B_ROW = G::B_ROW;
    using Fr = Frags<TM, TN>;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int tiles_m = (int)((f.M + BM - 1) / BM), tiles_n = (int)((f.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(bid, nblocks);
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
    // operands: whole rows of a slice, their chunks swizzled;
    // the others: 64 consecutive chunk positions of the slot.  Rows and
    // chunks past the edge read the last valid ones.
    const char* src[COPIES];
    int dst[COPIES];
#pragma unroll
    for (int i = 0; i < A_COPIES; ++i) {
        if constexpr (AMC) {
            const int j = wave * A_COPIES + i, q = 64 * j + lane, k = q / A_CHUNKS;
            int c = chunk_pos(q % A_CHUNKS, k);
            const int64_t left = (f.Mr - m0) / 8 - 1;
            c = c <= left ? c : (int)left;
            src[i] = A + ((int64_t)k * f.lda + m0 + 8 * c) * 2;
            dst[i] = j * 1024;
        } else {
            const int r0 = BM / 4 * wave + RPC * i, r = r0 + lane / RCH;
            const int c = lane % RCH ^ row_swz<BK>(r);
            src[i] = A + ((m0 + (r < mlim ? r : mlim - 1)) * f.lda + 8 * c) * 2;
            dst[i] = r0 * ROW;
        }
    }
#pragma unroll
    for (int i = 0; i < G::B_COPIES; ++i) {
        if constexpr (BKC) {
            const int r0 = BN / 4 * wave + RPC * i, r = r0 + lane / RCH;
            const int c = lane % RCH ^ row_swz<BK>(r);
            const bool second = DUAL && r >= G::OUT;
            int rr = second ? r - G::OUT : r;
            rr = rr < nlim ? rr : nlim - 1;
            src[A_COPIES + i] = B + (second ? b_diff : 0) + ((n0 + rr) * f.ldb + 8 * c) * 2;
            dst[A_COPIES + i] = A_BYTES + r0 * ROW;
        } else {
            const int j = wave * G::B_COPIES + i, q = 64 * j + lane, k = q / G::B_CHUNKS;
            int c = chunk_pos(q % G::B_CHUNKS, k);
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
    auto copy = [&](int s, int slot, int i) {
        copy_to_lds(src[i] + (i < A_COPIES ? a_at(j0 + s) : b_at(j0 + s)),
                    lds0 + (unsigned)slot * G::SLOT_BYTES + dst[i]);
    };

    // Fragment read offsets within a slot.
    int a_off[TM][KS][AMC ? 2 : 1], b_off[TN][KS][BKC ? 1 : 2];
    const int q4 = lane >> 4, t16 = lane & 15;
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (AMC) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 16 + 8 * (q4 >> 1) + 4 * h + (t16 >> 2);
                    const int m = G::WROWS * wm + 32 * t + 16 * (q4 & 1) + 4 * (t16 & 3);
                    a_off[t][ks][h] = k * A_KROW + (chunk_pos(m >> 3, k) << 4) + ((m & 7) << 1);
                }
            } else {
                const int r = G::WROWS * wm + 32 * t + (lane & 31);
                a_off[t][ks][0] = r * ROW + (((2 * ks + (lane >> 5)) ^ row_swz<BK>(r)) << 4);
            }
        }
#pragma unroll
    for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (BKC) {
                const int r = G::column(wn, t) + (lane & 31);
                b_off[t][ks][0] = A_BYTES + r * ROW + (((2 * ks + (lane >> 5)) ^ row_swz<BK>(r)) << 4);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = ks * 16 + 8 * (q4 >> 1) + 4 * h + (t16 >> 2);
                    const int n = G::column(wn, t) + 16 * (q4 & 1) + 4 * (t16 & 3);
                    b_off[t][ks][h] = A_BYTES + k * B_ROW + (chunk_pos(n >> 3, k) << 4) + ((n & 7) << 1);
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
    // Read r of K-step ks of a slot, in the order the next K-step needs them:
    // A0, B0 .. B(TN-1), A1 .. A(TM-1).
    auto read = [&](Fr& fr, int slot, int ks, int r) {
        const unsigned char* base = smem + slot * G::SLOT_BYTES;
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
    // beta * C goes into the sum first, so that the stores need no second read.
    if constexpr (STORE != STORE_PART && FORM == BLOCK_DW) {
        if (f.beta != 0.0f && f.ksplit == 1) {
            int64_t ld;
            const uint16_t* C = plane_of<FORM>(f, 0, bt, ld);
            const bool ok = vec4_ok(C, ld);
#pragma unroll
            for (int tm = 0; tm < TM; ++tm) {
                const int mi = G::WROWS * wm + 32 * tm + (lane & 31);
                if (mi >= mlim) continue;
#pragma unroll
                for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float c[4];
                        load4<DT>(C + (m0 + mi) * ld + n0, G::column(wn, tn) + 8 * q + 4 * (lane >> 5), nlim, ok, c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[tm][tn][4 * q + e] = in_acc(f.beta * c[e]);
                    }
            }
        }
    }

    // One K-step: the MFMAs on `use`, with the reads of (slot rs, K-step rks)
    // and the copies c0 .. c1-1 of slice cs (into slot cslot) spread between them.
    constexpr int NM = TM * TN, NR = TM + TN;
    auto kstep = [&](const Fr& use, Fr& nxt, bool do_read, int rs, int rks, bool do_copy, int cs, int cslot, int c0,
                     int c1) {
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            const int tm = i / TN, tn = (tm & 1) ? TN - 1 - i % TN : i % TN;
            acc[tm][tn] = mfma<DT>(use.b[tn], use.a[tm], acc[tm][tn]);
            if (do_copy) {
#pragma unroll
                for (int c = c0; c < c1; ++c)
                    if (i == (c - c0) * NM / (c1 - c0)) copy(cs, cslot, c);
            }
            if (do_read) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if ((r + 1 < NM ? r + 1 : NM - 1) == i) read(nxt, rs, rks, r);
            }
            fence_sched();
        }
    };

    // Prologue: request slices 0 .. AHEAD-1, make slice 0 visible, read its fragments.
    Fr fr[2];
    const int npro = nk < AHEAD ? nk : AHEAD;
    for (int s = 0; s < npro; ++s)
        for (int i = 0; i < COPIES; ++i) copy(s, s, i);
    if (nk > 0) {
        wait_slices<COPIES, AHEAD - 1>(npro - 1);
        slice_barrier();
#pragma unroll
        for (int r = 0; r < NR; ++r) read(fr[0], 0, 0, r);
    }
    // Slice j (slot cur): wait for this wave's copies of slice j+1 (later ones
    // may stay in flight), barrier (slice j+1 visible, the slot `old` of slice
    // j-1 free), then the K-steps, which read the next K-step's fragments and
    // issue the copies of slice j+AHEAD a few at a time.
    int j = 0, cur = 0, old = SLOTS - 1;
    for (; j + AHEAD < nk; ++j) {
        const int nxt = cur + 1 == SLOTS ? 0 : cur + 1;
        wait_vm<COPIES * (AHEAD - 2)>();
        slice_barrier();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            kstep(fr[ks & 1], fr[~ks & 1], true, ks + 1 < KS ? cur : nxt, (ks + 1) % KS, true, j + AHEAD, old,
                  ks * COPIES / KS, (ks + 1) * COPIES / KS);
        old = cur;
        cur = nxt;
    }
    for (; j < nk; ++j) {
        const int nxt = cur + 1 == SLOTS ? 0 : cur + 1;
        const bool next = j + 1 < nk;
        if (next) {
            wait_slices<COPIES, AHEAD - 2>(nk - j - 2);
            slice_barrier();
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            kstep(fr[ks & 1], fr[~ks & 1], ks + 1 < KS || next, ks + 1 < KS ? cur : nxt, (ks + 1) % KS, false, 0, 0, 0,
                  1);
        cur = nxt;
    }

    // Contraction tail: the range that ends at the last whole slice adds the
    // remaining K % BK of every segment, staged by ordinary loads into the
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
                    const int r = (is_a ? BM / 4 * wave + RPC * i : BN / 4 * wave + RPC * ib) + lane / RCH;
                    const int k = 8 * (lane % RCH ^ row_swz<BK>(r));
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
            for (int r = 0; r < NR; ++r) read(fr[0], 0, 0, r);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                kstep(fr[ks & 1], fr[~ks & 1], ks + 1 < KS, 0, (ks + 1) % KS, false, 0, 0, 0, 1);
        }
    }

    // Lane holds C(m, n..n+3), m = row within the 32x32 block.
    if (STORE == STORE_PART || (STORE == STORE_EITHER && f.ksplit > 1)) {
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
        return;
    }
    if constexpr (STORE != STORE_PART) {
        // Outputs go through LDS, 32 rows at a time in each wave's own piece: the
        // lane layout would store 16 bytes of each of 32 rows at once.  A wave's
        // LDS operations stay in order, so one piece serves all rows.
        __syncthreads();
        acc_settle();
        constexpr int NP = planes<FORM>(), PIECE = 32 * G::STAGE_ROW;
        unsigned char* st = smem + wave * NP * PIECE;
        const int wrow0 = G::WROWS * wm, wcol0 = G::WOUT * wn;       // this wave's corner of the tile
        const int cols = nlim - wcol0 < G::WOUT ? nlim - wcol0 : G::WOUT;
        uint16_t* corner[NP];
        int64_t ld[NP];
        bool vec[NP], keep[NP];
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) {
            uint16_t* C = plane_of<FORM>(f, pl, bt, ld[pl]);
            keep[pl] = C != nullptr;
            vec[pl] = ld[pl] % 8 == 0 && ((uintptr_t)C & 15) == 0;
            corner[pl] = C + (m0 + wrow0) * ld[pl] + n0 + wcol0;
        }
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            const int r0 = 32 * tm, fr = lane & 31, nq = 4 * (lane >> 5);
            const int rows = mlim - wrow0 - r0 < 32 ? mlim - wrow0 - r0 : 32;
            wave_fence();
            auto stage = [&](auto far) {
#pragma unroll
                for (int tn = 0; tn < G::TNO; ++tn)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        f32x4 g, u = f32x4{};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            g[e] = from_acc(acc[tm][tn][4 * q + e]);
                            if constexpr (DUAL) u[e] = from_acc(acc[tm][tn + TN - G::TNO][4 * q + e]);
                        }
                        const int c = 32 * tn + 8 * q + nq;
                        if constexpr (FORM == BLOCK_AGAIN) {
                            again_grad<DT>(f, m0 + wrow0 + r0 + fr, n0 + wcol0 + c, g, u);
                        }
#pragma unroll
                        for (int pl = 0; pl < NP; ++pl) {
                            float v[4];
                            block_value<DT, FORM, decltype(far)::value>(pl, g, u, v);
                            *(uint2*)(st + pl * PIECE + fr * G::STAGE_ROW + c * 2) =
                                make_uint2((uint32_t)to_bits<DT>(v[0]) | ((uint32_t)to_bits<DT>(v[1]) << 16),
                                           (uint32_t)to_bits<DT>(v[2]) | ((uint32_t)to_bits<DT>(v[3]) << 16));
                        }
                    }
            };
            if constexpr (FORM == BLOCK_FORWARD) {
                uint32_t bits = 0;
#pragma unroll
                for (int i = 0; i < G::TNO * 16; ++i) bits = max_bits(bits, from_acc(acc[tm][i / 16][i % 16]));
                with_far(any_far(bits), stage);
            } else {
                stage(std::false_type{});
            }
            wave_fence();
#pragma unroll
            for (int pl = 0; pl < NP; ++pl) {
                if (!keep[pl]) continue;
                const unsigned char* from = st + pl * PIECE;
                uint16_t* to = corner[pl] + r0 * ld[pl];
                if (vec[pl]) {
                    constexpr int CH = G::WOUT / 8, PER = 32 * CH / 64;      // 16-byte chunks of a row, per lane
                    u32x4 w[PER];
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        w[i] = *(const u32x4*)(from + (64 * i + lane) / CH * G::STAGE_ROW + (64 * i + lane) % CH * 16);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int r = (64 * i + lane) / CH, c = (64 * i + lane) % CH * 8;
                        if (r >= rows || c >= cols) continue;
                        uint16_t* o = to + r * ld[pl] + c;
                        if (c + 8 <= cols) {
                            *(u32x4*)o = w[i];
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (c + e < cols) o[e] = (uint16_t)(w[i][e / 2] >> (16 * (e & 1)));
                        }
                    }
                } else {
                    // Rows that are not 16-byte aligned: consecutive elements by consecutive lanes.
                    for (int r = 0; r < rows; ++r)
                        for (int c = lane; c < cols; c += 64)
                            to[r * ld[pl] + c] = *(const uint16_t*)(from + r * G::STAGE_ROW + c * 2);
                }
            }
            fence_sched();
        }
    }
}

template <int DT, int FORM, int T, bool AMC, bool BKC, int STORE>
__global__ __launch_bounds__(NT, 1) void k_block(BlockArgs f) {
    extern __shared__ __align__(16) unsigned char smem[];
    block_body<DT, FORM, T, AMC, BKC, STORE>(f, blockIdx.x, gridDim.x, smem);
}

// Second phase of a split: one thread per 16-byte chunk of a tile's
// accumulators sums the ranges in range order and stores four outputs.
template <int DT, int FORM, int T>
__device__ __forceinline__ void reduce_body(const BlockArgs& f, int bid, int nblocks) {
    using G = Cfg<FORM, T>;
    constexpr int BM = T;
    constexpr int TM = G::TM, TN = G::TN, TNO = G::TNO, CH = TM * TNO * 4;
    constexpr int64_t TILE = (int64_t)NT * TM * TN * 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    const int tiles_m = (int)((f.M + BM - 1) / BM), tiles_n = (int)((f.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(bid, nblocks);
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
    const int ni = G::WOUT * wn + 32 * tn + 8 * q + 4 * (lane >> 5);
    if (m >= f.M || ni >= nlim) return;
    const float* part = f.part + (int64_t)tile * f.ksplit * TILE + 4 * tid;
    auto sum = [&](int chunk) {
        const float* p = part + (int64_t)chunk * NT * 4;
        f32x4 a = *(const f32x4*)p;
        // Eight ranges are requested at a time and added one by one.
        for (int s = 1; s < f.ksplit; s += 8) {
            f32x4 b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = s + i < f.ksplit ? *(const f32x4*)(p + (s + i) * TILE) : f32x4{};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (s + i < f.ksplit) a = a + b[i];
        }
        return a;
    };
    f32x4 g = sum((tm * TN + tn) * 4 + q);
    f32x4 u = G::DUAL ? sum((tm * TN + tn + TNO) * 4 + q) : g;
    if constexpr (FORM == BLOCK_AGAIN) {
        again_grad<DT>(f, m, n0 + ni, g, u);
    }
#pragma unroll
    for (int plane = 0; plane < planes<FORM>(); ++plane) {
        int64_t ld;
        uint16_t* C = plane_of<FORM>(f, plane, bt, ld);
        if (FORM == BLOCK_FORWARD && C == nullptr) continue;
        float v[4];
        if (FORM == BLOCK_FORWARD && plane == 0)
            gated_product4<DT>({g[0], g[1], g[2], g[3]}, {u[0], u[1], u[2], u[3]}, v);
        else block_value<DT, FORM, false>(plane, g, u, v);
        store_out4<DT, EPI_NONE>(C + m * ld + n0, ni, nlim, vec4_ok(C, ld), f.beta, v);
    }
}

template <int DT, int FORM, int T>
__global__ __launch_bounds__(NT) void k_block_reduce(BlockArgs f) {
    reduce_body<DT, FORM, T>(f, blockIdx.x, gridDim.x);
}

// Fills in the ranges and returns the workgroups of a launch with ks of them.
template <int FORM, int T>
int64_t set_ranges(BlockArgs& a, int ks) {
    using G = Cfg<FORM, T>;
    const int64_t slices = (a.K / G::BK) * (FORM == BLOCK_DX ? 2 : 1);
    a.nks = (int)(ks > 1 ? (slices + ks - 1) / ks : (slices > 0 ? slices : 1));
    a.ksplit = ks > 1 ? (int)((slices + a.nks - 1) / a.nks) : 1;
    return ((a.M + T - 1) / T) * a.batches_m * (((a.N + G::OUT - 1) / G::OUT) * a.batches_n) * a.ksplit;
}
// Workgroups of the second phase, per tile.
template <int FORM, int T>
constexpr int reduce_chunks() {
    using G = Cfg<FORM, T>;
    return G::TM * G::TNO * 4;
}

template <int DT, int FORM, int T, bool AMC, bool BKC>
hipError_t launch_block(BlockArgs a, int ks, hipStream_t s) {
    using G = Cfg<FORM, T>;
    const int64_t wgs = set_ranges<FORM, T>(a, ks);
    auto go = [&](auto kern, bool (&done)[MAX_DEVICES]) -> hipError_t {
        if (hipError_t e = set_lds_limit_once((const void*)kern, G::LDS, done); e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(NT), G::LDS, s, a);
        return hipGetLastError();
    };
    if (a.ksplit == 1) {
        static bool done[MAX_DEVICES] = {};
        return go(k_block<DT, FORM, T, AMC, BKC, STORE_OUT>, done);
    }
    static bool done[MAX_DEVICES] = {};
    if (hipError_t e = go(k_block<DT, FORM, T, AMC, BKC, STORE_PART>, done); e != hipSuccess) return e;
    hipLaunchKernelGGL((k_block_reduce<DT, FORM, T>),
                       dim3((unsigned)(wgs / a.ksplit * reduce_chunks<FORM, T>())), dim3(NT), 0, s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace mgemm
