// Products of microscaled 4-bit codes for gfx950:
//     C(m,n) = alpha * sum_j 2^(sa[m][j] + sb[n][j] - 254) * sum_{k in block j} qa[m][k] qb[n][k] + beta * C(m,n)
// with both code matrices K-contiguous (qb holds the weights one output
// column per row), and the gated pair Z = SiLU(A Bg^T) * (A Bu^T).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 on E2M1 operands takes from each lane one
// 32-element block of one row (16 bytes) and one scale byte, so a lane's
// fragment is exactly one block of the format and the scaling costs no
// instruction of its own; sums are FP32.  It does 64 k in the 32 cycles in
// which the BF16 instruction does 16, and a 128-element slice of a row is 64
// bytes, the bytes of a 32-element BF16 slice.  The tile loop is therefore
// that of k_h_dma.hip byte for byte: a four-slot direct-to-LDS ring, 64-byte
// rows with their 16-byte chunks swizzled, two K-steps per slice, fragments
// read one K-step ahead, one barrier per slice, with the L2 and LDS traffic per
// matrix instruction of the BF16 kernel.
//
// Scales come as 16 bytes per row (four slices, 512 k), staged into a
// two-slot LDS ring of their own with every fourth slice: a copy of four
// bytes per row with every slice would touch as many cache lines as the codes'
// copies do.  A lane reads its row's dword of four scales per
// slice and shifts it so that the byte its half of the wave needs is
// selected by the instruction's byte select (0 in the first K-step, 2 in the
// second).
//
// Measured (codes given, calls back to back, over several cards): 8192 x 12288 x
// 4096 296 to 303 us (2.7 to 2.8 PFLOP/s; in a kernel trace behind the quantisation of
// 8192 rows 326 at least and 344 in the median), 8192 x 4096 x 12288 254 to 260 (3.2),
// 4096^3 53 to 55; the gated pair 1024 x 12288 x 4096 84 to 88 (the call, with 6 of
// quantisation, 90 to 94; traced 95 to 97).  A slice of a 256x256 tile
// takes 2740 cycles for 1024 of matrix work (34.6 cycles an instruction alone):
// 2580 without the scales' copies, 2230 without their LDS reads too, 2180 with
// constant scales, so the codes' copies bound it and the scales add a quarter.
// Pairs of slices requested together (whole 128-byte lines, a five-slot ring of
// 256x192 tiles), two scale dwords to a read and 16 scale bytes kept in
// registers were each built and timed: no faster, the last one slower.
//
// Restrictions (host-checked): code rows 16-byte aligned, scale rows 16-byte
// aligned with a stride that is a multiple of 16 (the last group of a row is
// read whole).  k_mx4_general takes the rest.
#include "mx4.h"

namespace mgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int NT = 256;
constexpr int BK = 128;                          // elements per slice
constexpr int ROW = BK / 2;                      // bytes per operand row per slice
constexpr int SLOTS = 4, AHEAD = SLOTS - 1;      // slices in flight
constexpr int SCALE_ROW = 16, GROUP = 4;         // scale bytes per row and group of GROUP slices
constexpr int SPLIT_GROUP_M = 2, UNSPLIT_GROUP_M = 4;   // tile orders of k_h_dma.hip

// Plain products: four waves 2x2, BM/2 x BN/2 each.  The gated pair: 96 rows
// of each B matrix in the 192-row B slot, four waves of BM/4 x 192, so a wave
// holds G and U of the same outputs in matching registers.
template <int BN, int BM, bool DUAL>
struct Cfg {
    static_assert(BN == 256 || BN == 192, "tile width");
    static_assert(!DUAL || BN == 192, "the gated pair uses the 192-wide slot");
    static constexpr int A_BYTES = BM * ROW, SLOT_BYTES = (BM + BN) * ROW;
    static constexpr int A_COPIES = BM / 64, B_COPIES = BN / 64;     // 1 KiB copies per wave per slice
    static constexpr int COPIES = A_COPIES + B_COPIES;
    static constexpr int S_ROWS = BM + BN;                           // scale rows per group
    static constexpr int S_COPIES = (S_ROWS / 64 + 3) / 4;           // 1 KiB copies per wave per group
    static constexpr int S_BYTES = S_ROWS * SCALE_ROW;
    static constexpr int LDS = SLOTS * SLOT_BYTES + 2 * S_BYTES;
    static constexpr int WROWS = DUAL ? BM / 4 : BM / 2;
    static constexpr int TM = WROWS / 32, TN = DUAL ? BN / 32 : BN / 64;
    static constexpr int WN = DUAL ? 0 : BN / 2;
    static constexpr int OUT = DUAL ? BN / 2 : BN;
};

__device__ __forceinline__ int swz(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }

template <int N>
__device__ __forceinline__ void wait_vm() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
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

// c + x y^T on E2M1 blocks (formats 4), the scale of K-step ks in byte 2*ks.
template <int KS>
__device__ __forceinline__ f32x16 mfma4(i32x4 x, i32x4 y, f32x16 c, int sx, int sy) {
    const i32x8 xa = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 ya = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xa, ya, c, 4, 4, 2 * KS, sx, 2 * KS, sy);
}

template <int TM, int TN>
struct Frags {
    i32x4 a[TM];
    i32x4 b[TN];
};
template <int TM, int TN>
struct Scales {
    int a[TM];
    int b[TN];
};

template <int CT, int BN, int BM, bool DUAL, bool PARTIAL>
__global__ __launch_bounds__(NT, 1) void k_mx4_dma(Problem p, Mx4Args f) {
    using G = Cfg<BN, BM, DUAL>;
    constexpr int TM = G::TM, TN = G::TN, COPIES = G::COPIES, A_COPIES = G::A_COPIES;
    constexpr int S_COPIES = G::S_COPIES;
    using Fr = Frags<TM, TN>;
    using Sc = Scales<TM, TN>;
    extern __shared__ __align__(16) unsigned char smem[];
    const ClockStamp stamp0 = clock_stamp_begin();
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = DUAL ? wave : wave >> 1, wn = DUAL ? 0 : wave & 1;
    const int tiles_m = (int)((p.M + BM - 1) / BM), tiles_n = (int)((p.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(blockIdx.x, gridDim.x);
    const int split = pos % f.ksplit;
    int tmi, tni;
    tile_from_linear(pos / f.ksplit, tiles_m, tiles_n, f.ksplit > 1 ? SPLIT_GROUP_M : UNSPLIT_GROUP_M, tmi, tni);
    const int64_t m0 = (int64_t)tmi * BM, n0 = (int64_t)tni * G::OUT;
    const int mlim = (int)(p.M - m0 < BM ? p.M - m0 : BM);
    const int nlim = (int)(p.N - n0 < G::OUT ? p.N - n0 : G::OUT);
    const int blocks = (int)((p.K + MX_BLOCK - 1) / MX_BLOCK);
    const int nk_all = blocks / 4;                       // whole slices
    const int j0 = split * f.nks;                        // this range's first slice
    const int nk = nk_all - j0 < f.nks ? nk_all - j0 : f.nks;

    // Row r of the B slot: an output column's codes, the last valid row past the edge.
    auto b_codes = [&](int r) -> const uint8_t* {
        if constexpr (DUAL) {
            const bool second = r >= BN / 2;
            int rr = second ? r - BN / 2 : r;
            rr = rr < nlim ? rr : nlim - 1;
            return (const uint8_t*)(second ? p.B2 : p.B) + (n0 + rr) * p.ldb;
        } else {
            return (const uint8_t*)p.B + (n0 + (r < nlim ? r : nlim - 1)) * p.ldb;
        }
    };
    auto b_scales = [&](int r) -> const uint8_t* {
        if constexpr (DUAL) {
            const bool second = r >= BN / 2;
            int rr = second ? r - BN / 2 : r;
            rr = rr < nlim ? rr : nlim - 1;
            return (second ? f.sb2 : f.sb) + (n0 + rr) * f.ldsb;
        } else {
            return f.sb + (n0 + (r < nlim ? r : nlim - 1)) * f.ldsb;
        }
    };
    // Copies of this wave: 16 rows each, lane l takes row l/4's chunk
    // (l%4 ^ swz) so that it lands swizzled.
    const uint8_t* src[COPIES];
    int dst[COPIES];
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
        const bool is_a = i < A_COPIES;
        const int r = is_a ? BM / 4 * wave + 16 * i + (lane >> 2) : BN / 4 * wave + 16 * (i - A_COPIES) + (lane >> 2);
        const int c = (lane & 3) ^ swz(r);
        const uint8_t* row = is_a ? (const uint8_t*)p.A + (m0 + (r < mlim ? r : mlim - 1)) * p.lda : b_codes(r);
        src[i] = row + (int64_t)j0 * ROW + 16 * c;
        dst[i] = (is_a ? 0 : G::A_BYTES) + (is_a ? BM / 4 * wave + 16 * i : BN / 4 * wave + 16 * (i - A_COPIES)) * ROW;
    }
    // Scale copies: 64 rows each (lane l: row l's 16 bytes); a wave whose
    // share runs past the last 64 rows repeats the last copy.
    const uint8_t* ssrc[S_COPIES];
    int sdst[S_COPIES];
#pragma unroll
    for (int i = 0; i < S_COPIES; ++i) {
        int j = wave * S_COPIES + i;
        j = j < G::S_ROWS / 64 ? j : G::S_ROWS / 64 - 1;
        const int r = 64 * j + lane;
        ssrc[i] = r < BM ? f.sa + (m0 + (r < mlim ? r : mlim - 1)) * f.ldsa : b_scales(r - BM);
        sdst[i] = SLOTS * G::SLOT_BYTES + 64 * j * SCALE_ROW;
    }
    const unsigned lds0 = (unsigned)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
    auto copy = [&](int s, int i) {
        copy_to_lds(src[i] + (int64_t)s * ROW, lds0 + (unsigned)(s % SLOTS) * G::SLOT_BYTES + dst[i]);
    };
    // Whether slice s (of this range) brings its group's scales with it, and the copies that it then is.
    auto brings = [&](int s) { return s == 0 || ((j0 + s) & (GROUP - 1)) == 0; };
    auto copy_scales = [&](int s) {
        const int g = (j0 + s) / GROUP;
#pragma unroll
        for (int i = 0; i < S_COPIES; ++i)
            copy_to_lds(ssrc[i] + (int64_t)g * SCALE_ROW, lds0 + (unsigned)((g & 1) * G::S_BYTES) + sdst[i]);
    };
    // Waits until only the copies of slice s (if any) are still in flight.
    auto wait_but = [&](int s) {
        if (s >= nk) wait_vm<0>();
        else if (brings(s)) wait_vm<COPIES + S_COPIES>();
        else wait_vm<COPIES>();
    };

    int a_off[TM][2], b_off[TN][2], sa_off[TM], sb_off[TN];
#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int r = G::WROWS * wm + 32 * t + (lane & 31);
        sa_off[t] = SLOTS * G::SLOT_BYTES + r * SCALE_ROW;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) a_off[t][ks] = r * ROW + (((2 * ks + (lane >> 5)) ^ swz(r)) << 4);
    }
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        const int r = G::WN * wn + 32 * t + (lane & 31);
        sb_off[t] = SLOTS * G::SLOT_BYTES + (BM + r) * SCALE_ROW;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            b_off[t][ks] = G::A_BYTES + r * ROW + (((2 * ks + (lane >> 5)) ^ swz(r)) << 4);
    }
    // Read r of (slice s, K-step ks): A0, B0 .. B(TN-1), A1 .. A(TM-1).
    auto read = [&](Fr& fr, int s, int ks, int r) {
        const unsigned char* base = smem + (s % SLOTS) * G::SLOT_BYTES;
        if (r == 0) fr.a[0] = *(const i32x4*)(base + a_off[0][ks]);
        else if (r <= TN) fr.b[r - 1] = *(const i32x4*)(base + b_off[r - 1][ks]);
        else fr.a[r - TN] = *(const i32x4*)(base + a_off[r - TN][ks]);
    };
    const int half = 8 * (lane >> 5);
    auto read_scale = [&](Sc& sc, int s, int r) {
        const int j = j0 + s;
        const unsigned char* base = smem + ((j / GROUP) & 1) * G::S_BYTES + 4 * (j & (GROUP - 1));
        if (r < TM) sc.a[r] = *(const int*)(base + sa_off[r]);
        else sc.b[r - TM] = *(const int*)(base + sb_off[r - TM]);
    };
    auto shift_scales = [&](Sc& sc) {
#pragma unroll
        for (int t = 0; t < TM; ++t) sc.a[t] = (int)((unsigned)sc.a[t] >> half);
#pragma unroll
        for (int t = 0; t < TN; ++t) sc.b[t] = (int)((unsigned)sc.b[t] >> half);
    };

    f32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

    // One K-step: the MFMAs on `use`; the reads of (rs, rks) and the copies
    // c0 .. c1-1 of slice cs are spread between them, and in the second
    // K-step of a slice the next slice's scales too.
    constexpr int NM = TM * TN, NR = TM + TN;
    auto kstep = [&](auto KS, const Fr& use, const Sc& sc, Fr& nxt, Sc& snxt, bool do_read, int rs, int rks,
                     bool do_copy, int cs, int c0, int c1) {
        constexpr int ks = decltype(KS)::value;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            const int tm = i / TN, tn = (tm & 1) ? TN - 1 - i % TN : i % TN;
            acc[tm][tn] = mfma4<ks>(use.b[tn], use.a[tm], acc[tm][tn], sc.b[tn], sc.a[tm]);
            if (do_copy) {
#pragma unroll
                for (int c = c0; c < c1; ++c)
                    if (i == (c - c0) * NM / (c1 - c0)) copy(cs, c);
            }
            if (do_read) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (r * NM / NR == i) {
                        read(nxt, rs, rks, r);
                        if constexpr (ks == 1) read_scale(snxt, rs, r);
                    }
            }
            fence_sched();
        }
        if (ks == 1 && do_read) shift_scales(snxt);
    };
    constexpr std::integral_constant<int, 0> K0{};
    constexpr std::integral_constant<int, 1> K1{};

    // Prologue: request slices 0 .. AHEAD-1, make slice 0 visible, read its first fragments.
    Fr f0, f1;
    Sc s0, s1;
    const int npro = nk < AHEAD ? nk : AHEAD;
    for (int s = 0; s < npro; ++s) {
        if (brings(s)) copy_scales(s);
        for (int i = 0; i < COPIES; ++i) copy(s, i);
    }
    if (nk > 0) {
        // Slices 1 and 2 may stay in flight: only one of them can bring scales.
        if (npro == 3) {
            if (brings(1) || brings(2)) wait_vm<2 * COPIES + S_COPIES>();
            else wait_vm<2 * COPIES>();
        } else {
            wait_but(1);
        }
        slice_barrier();
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            read(f0, 0, 0, r);
            read_scale(s0, 0, r);
        }
        shift_scales(s0);
    }
    // Slice j: wait for this wave's copies of slice j+1 (slice j+2 may stay
    // in flight), barrier (slice j+1 visible, the slot of slice j-1 free),
    // then K-step 0 with the A copies of slice j+AHEAD and K-step 1 with its
    // B copies.  Scales alternate between s0 and s1.  The scale slot that a
    // group overwrites was last read two groups ago.
    auto slice = [&](int j, Sc& sc, Sc& sn) {
        const bool next = j + 1 < nk, more = j + AHEAD < nk;
        if (next) {
            wait_but(j + 2);
            slice_barrier();
        }
        if (more && brings(j + AHEAD)) copy_scales(j + AHEAD);
        kstep(K0, f0, sc, f1, sn, true, j, 1, more, j + AHEAD, 0, A_COPIES);
        kstep(K1, f1, sc, f0, sn, next, j + 1, 0, more, j + AHEAD, A_COPIES, COPIES);
    };
    int j = 0;
    for (; j + 1 < nk; j += 2) {
        slice(j, s0, s1);
        slice(j + 1, s1, s0);
    }
    if (j < nk) slice(j, s0, s1);

    // K tail: the range that ends at the last whole slice adds the remaining
    // 1 to 3 blocks of each row, staged by ordinary loads into the positions
    // that the copies fill, with zero codes and scale 1 for the blocks that
    // do not exist.  No copy is in flight any more.
    const int btail = blocks - 4 * nk_all;
    if (btail > 0 && j0 + nk == nk_all) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const int r = i < A_COPIES ? BM / 4 * wave + 16 * i + (lane >> 2)
                                       : BN / 4 * wave + 16 * (i - A_COPIES) + (lane >> 2);
            i32x4 v = i32x4{0, 0, 0, 0};
            if (((lane & 3) ^ swz(r)) < btail) v = *(const i32x4*)(src[i] + (int64_t)nk * ROW);
            *(i32x4*)(smem + dst[i] + 16 * lane) = v;
        }
#pragma unroll
        for (int i = 0; i < S_COPIES; ++i) {
            uint32_t w = 0x7F7F7F7Fu;
#pragma unroll
            for (int b = 0; b < 3; ++b)
                if (b < btail) w = (w & ~(255u << (8 * b))) | ((uint32_t)ssrc[i][4 * (int64_t)nk_all + b] << (8 * b));
            *(uint32_t*)(smem + sdst[i] + lane * SCALE_ROW) = w;
        }
        __syncthreads();
        // Slot 0 of both rings: read as slice 0 with the scales at dword 0.
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            read(f0, 0, 0, r);
            read(f1, 0, 1, r);
        }
#pragma unroll
        for (int t = 0; t < TM; ++t) s0.a[t] = *(const int*)(smem + sa_off[t]);
#pragma unroll
        for (int t = 0; t < TN; ++t) s0.b[t] = *(const int*)(smem + sb_off[t]);
        shift_scales(s0);
        kstep(K0, f0, s0, f1, s1, false, 0, 0, false, 0, 0, 1);
        kstep(K1, f1, s0, f0, s1, false, 0, 0, false, 0, 0, 1);
    }

    // Epilogue: lane holds C(m, n..n+3), m = row within the 32x32 block.
    if constexpr (PARTIAL) {
        float* dstp = f.part + ((int64_t)(tmi * tiles_n + tni) * f.ksplit + split) * (int64_t)(NT * TM * TN * 16) +
                      4 * tid;
#pragma unroll
        for (int tm = 0; tm < TM; ++tm) {
            if (G::WROWS * wm + 32 * tm + (lane & 31) >= mlim) continue;
#pragma unroll
            for (int tn = 0; tn < TN; ++tn)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16& a = acc[tm][tn];
                    *(f32x4*)(dstp + (int64_t)((tm * TN + tn) * 4 + q) * NT * 4) =
                        f32x4{a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
                }
        }
        clock_stamp_end(p, stamp0);
        return;
    }
    const bool vec_ok = mx4_vec_ok<CT>(p.C, p.ldc);
    const int fr = lane & 31, nq = 4 * (lane >> 5);
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
        const int mi = G::WROWS * wm + 32 * tm + fr;
        if (mi >= mlim) continue;
        const int64_t row = (m0 + mi) * p.ldc + n0;
        auto store = [&](auto far) {
#pragma unroll
            for (int tn = 0; tn < (DUAL ? TN / 2 : TN); ++tn)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if constexpr (DUAL)
                            v[e] = gated_product<CT, far>(acc[tm][tn][4 * q + e], acc[tm][tn + TN / 2][4 * q + e]);
                        else v[e] = p.alpha * acc[tm][tn][4 * q + e];
                    }
                    mx4_store4<CT>(p.C, row, G::WN * wn + 32 * tn + 8 * q + nq, nlim, vec_ok, p.beta, v);
                }
        };
        if constexpr (DUAL) {
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < TN / 2 * 16; ++i) bits = max_bits(bits, acc[tm][i / 16][i % 16]);
            with_far(any_far(bits), store);
        } else {
            store(std::false_type{});
        }
    }
    clock_stamp_end(p, stamp0);
}

// Second split-K phase: one thread per 16-byte chunk of a tile's
// accumulators sums the K ranges in range order and stores four outputs as
// the one-phase epilogue would.
template <int CT, int BN, int BM, bool DUAL>
__global__ __launch_bounds__(NT) void k_mx4_reduce(Problem p, Mx4Args f) {
    using G = Cfg<BN, BM, DUAL>;
    constexpr int TM = G::TM, TN = G::TN, TNO = DUAL ? TN / 2 : TN, CH = TM * TNO * 4;
    constexpr int64_t TILE = (int64_t)NT * TM * TN * 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = DUAL ? wave : wave >> 1, wn = DUAL ? 0 : wave & 1;
    const int tiles_m = (int)((p.M + BM - 1) / BM), tiles_n = (int)((p.N + G::OUT - 1) / G::OUT);
    const int pos = xcd_linear(blockIdx.x, gridDim.x);
    const int t = pos / CH, c = pos % CH;
    int tmi, tni;
    tile_from_linear(t, tiles_m, tiles_n, SPLIT_GROUP_M, tmi, tni);
    const int tm = c / (TNO * 4), tn = (c / 4) % TNO, q = c % 4;
    const int64_t m0 = (int64_t)tmi * BM, n0 = (int64_t)tni * G::OUT;
    const int mlim = (int)(p.M - m0 < BM ? p.M - m0 : BM);
    const int nlim = (int)(p.N - n0 < G::OUT ? p.N - n0 : G::OUT);
    const int mi = G::WROWS * wm + 32 * tm + (lane & 31);
    const int ni = G::WN * wn + 32 * tn + 8 * q + 4 * (lane >> 5);
    if (mi >= mlim || ni >= nlim) return;
    const float* tile = f.part + (int64_t)(tmi * tiles_n + tni) * f.ksplit * TILE + 4 * tid;
    auto sum = [&](int chunk) {
        const float* src = tile + (int64_t)chunk * NT * 4;
        f32x4 a = *(const f32x4*)src;
        // Eight ranges are requested at a time and added one by one.
        for (int s = 1; s < f.ksplit; s += 8) {
            f32x4 b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) b[i] = s + i < f.ksplit ? *(const f32x4*)(src + (s + i) * TILE) : f32x4{};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (s + i < f.ksplit) a = a + b[i];
        }
        return a;
    };
    const f32x4 g = sum((tm * TN + tn) * 4 + q);
    float v[4];
    if constexpr (DUAL) {
        const f32x4 u = sum((tm * TN + tn + TN / 2) * 4 + q);
        gated_product4<CT>({g[0], g[1], g[2], g[3]}, {u[0], u[1], u[2], u[3]}, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p.alpha * g[e];
    }
    mx4_store4<CT>(p.C, (m0 + mi) * p.ldc + n0, ni, nlim, mx4_vec_ok<CT>(p.C, p.ldc), p.beta, v);
}

// Any alignment and stride: 64x64 output tiles, one block of 32 per step
// decoded to FP32 in LDS, a 4x4 register block per thread.  A block's products
// are multiples of 1/4 up to 36, so its sum is exact; both scales are applied to
// the sum in one step, because a value times its own scale alone leaves FP32's
// range from scale byte 253 on while the product may lie well inside it.
//
// Bound by its FP32 arithmetic, byte loads and, for few rows, idle CUs: 2880 x 2880
// weights with packed scale rows of 90 bytes 235 / 247 / 335 us for 1 / 64 / 1024 rows,
// the gated pair 673 / 650 / 600.
constexpr int GT = 64;

template <int CT, bool DUAL>
__global__ __launch_bounds__(NT) void k_mx4_general(Problem p, Mx4Args f) {
    constexpr int NB = DUAL ? 2 : 1;
    __shared__ float As[MX_BLOCK][GT + 4];
    __shared__ float Bs[NB][MX_BLOCK][GT + 4];
    __shared__ int Ea[GT], Eb[NB][GT];                     // scale bytes of the block
    const int tid = threadIdx.x;
    const int tiles_n = (int)((p.N + GT - 1) / GT);
    const int64_t m0 = (int64_t)(blockIdx.x / tiles_n) * GT, n0 = (int64_t)(blockIdx.x % tiles_n) * GT;
    const int r = tid >> 2, part = tid & 3;                // staged row and its 8-code part
    const int tx = tid & 15, ty = tid >> 4;
    float acc[NB][4][4] = {};
    auto stage = [&](const void* codes, int64_t ld, const uint8_t* scales, int64_t lds, int64_t row, int64_t rows,
                     int64_t b, float (*to)[GT + 4], int* exps) {
        uint32_t w = 0, sc = 127;
        if (row < rows) {
            const uint8_t* q = (const uint8_t*)codes + row * ld + b * 16 + part * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) w |= (uint32_t)q[e] << (8 * e);
            sc = scales[row * lds + b];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) to[part * 8 + e][r] = mx4_value(w >> (4 * e));
        if (part == 0) exps[r] = (int)sc;
    };
    const int64_t blocks = (p.K + MX_BLOCK - 1) / MX_BLOCK;
    for (int64_t b = 0; b < blocks; ++b) {
        stage(p.A, p.lda, f.sa, f.ldsa, m0 + r, p.M, b, As, Ea);
        stage(p.B, p.ldb, f.sb, f.ldsb, n0 + r, p.N, b, Bs[0], Eb[0]);
        if constexpr (DUAL) stage(p.B2, p.ldb, f.sb2, f.ldsb, n0 + r, p.N, b, Bs[1], Eb[1]);
        __syncthreads();
        float sum[NB][4][4] = {};
#pragma unroll 4
        for (int k = 0; k < MX_BLOCK; ++k)
#pragma unroll
            for (int h = 0; h < NB; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sum[h][i][j] = fmaf(As[k][ty * 4 + i], Bs[h][k][tx * 4 + j], sum[h][i][j]);
#pragma unroll
        for (int h = 0; h < NB; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int ea = Ea[ty * 4 + i], eb = Eb[h][tx * 4 + j];
                    const float v = __builtin_amdgcn_ldexpf(sum[h][i][j], ea + eb - 254);
                    acc[h][i][j] += ea == 255 || eb == 255 ? __uint_as_float(0x7FC00000u) : v;
                }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= p.M) continue;
        float v[4];
        if constexpr (DUAL) {
            gated_product4<CT>(acc[0][i], acc[1][i], v);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = p.alpha * acc[0][i][j];
        }
        const int nlim = (int)(p.N - n0 < GT ? p.N - n0 : GT);
        mx4_store4<CT>(p.C, m * p.ldc + n0, tx * 4, nlim, mx4_vec_ok<CT>(p.C, p.ldc), p.beta, v);
    }
}

template <int CT, int BN, int BM, bool DUAL>
hipError_t launch_tiles(const Problem& p, Mx4Args a, int ksplit, const Workspace& ws, hipStream_t s) {
    using G = Cfg<BN, BM, DUAL>;
    const int nk = (int)(mx4_blocks(p.K) / 4);
    a.part = (float*)ws.part;
    a.nks = ksplit > 1 ? (nk + ksplit - 1) / ksplit : (nk > 0 ? nk : 1);
    a.ksplit = ksplit > 1 ? (nk + a.nks - 1) / a.nks : 1;
    const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + G::OUT - 1) / G::OUT);
    auto go = [&](auto kern, bool (&done)[MAX_DEVICES]) -> hipError_t {
        if (hipError_t e = set_lds_limit_once((const void*)kern, G::LDS, done); e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)(tiles * a.ksplit)), dim3(NT), G::LDS, s, p, a);
        return hipGetLastError();
    };
    if (a.ksplit == 1) {
        static bool done[MAX_DEVICES] = {};
        return go(k_mx4_dma<CT, BN, BM, DUAL, false>, done);
    }
    static bool done[MAX_DEVICES] = {};
    if (hipError_t e = go(k_mx4_dma<F32, BN, BM, DUAL, true>, done); e != hipSuccess) return e;
    constexpr int CH = G::TM * (DUAL ? G::TN / 2 : G::TN) * 4;
    hipLaunchKernelGGL((k_mx4_reduce<CT, BN, BM, DUAL>), dim3((unsigned)(tiles * CH)), dim3(NT), 0, s, p, a);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_ct(const Problem& p, const Mx4Args& a, int bn, int bm, int ksplit, const Workspace& ws,
                     hipStream_t s) {
    if (p.B2 != nullptr) {
        if (bm == 256) return launch_tiles<CT, 192, 256, true>(p, a, ksplit, ws, s);
        return launch_tiles<CT, 192, 128, true>(p, a, ksplit, ws, s);
    }
    if (bn == 256) return launch_tiles<CT, 256, 256, false>(p, a, ksplit, ws, s);
    if (bm == 256) return launch_tiles<CT, 192, 256, false>(p, a, ksplit, ws, s);
    if (bm == 128) return launch_tiles<CT, 192, 128, false>(p, a, ksplit, ws, s);
    return launch_tiles<CT, 192, 64, false>(p, a, ksplit, ws, s);
}

}  // namespace

bool mx4_mfma_supports(const Problem& p, const Mx4Args& a, int bn, int bm) {
    const bool dual = p.B2 != nullptr;
    if (bn == 256 ? (bm != 256 || dual) : bn != 192) return false;
    if (bm != 256 && bm != 128 && (bm != 64 || dual)) return false;
    auto al = [](const void* q) { return ((uintptr_t)q & 15) == 0; };
    if (p.lda % 16 != 0 || p.ldb % 16 != 0 || !al(p.A) || !al(p.B) || !al(p.B2)) return false;
    if (a.ldsa % 16 != 0 || a.ldsb % 16 != 0 || !al(a.sa) || !al(a.sb) || !al(a.sb2)) return false;
    if (mx4_blocks(p.K) > 0x3fffffff) return false;
    const int out = dual ? 96 : bn;
    const int64_t tiles = ((p.M + bm - 1) / bm) * ((p.N + out - 1) / out);
    return tiles > 0 && tiles <= 0x7fffffff / 64;
}

int mx4_splits(const Problem& p, int bn, int bm, int requested, const Workspace& ws) {
    const int out = p.B2 != nullptr ? 96 : bn;
    const int64_t tiles = ((p.M + bm - 1) / bm) * ((p.N + out - 1) / out);
    const int64_t nk = mx4_blocks(p.K) / 4;
    if (requested <= 1 || nk < 2) return 1;
    int64_t ks = requested < nk ? requested : nk;
    const int64_t nks = (nk + ks - 1) / ks;
    ks = (nk + nks - 1) / nks;
    const int64_t tile_bytes = (int64_t)bm * bn * 4;
    if (ws.part == nullptr || tiles * ks * tile_bytes > ws.part_bytes) return 0;
    return (int)ks;
}

hipError_t launch_mx4_mfma(const Problem& p, Mx4Args a, int bn, int bm, int ksplit, const Workspace& ws,
                           hipStream_t s) {
    if (p.dtype == F32) return launch_ct<F32>(p, a, bn, bm, ksplit, ws, s);
    if (p.dtype == F16) return launch_ct<F16>(p, a, bn, bm, ksplit, ws, s);
    return launch_ct<BF16>(p, a, bn, bm, ksplit, ws, s);
}

hipError_t launch_mx4_general(const Problem& p, const Mx4Args& a, hipStream_t s) {
    const int64_t tiles = ((p.M + GT - 1) / GT) * ((p.N + GT - 1) / GT);
    if (tiles > 0x7fffffff) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles);
    const bool dual = p.B2 != nullptr;
#define MX4_GENERAL(CT)                                                                                       \
    if (dual) hipLaunchKernelGGL((k_mx4_general<CT, true>), grid, dim3(NT), 0, s, p, a);                      \
    else hipLaunchKernelGGL((k_mx4_general<CT, false>), grid, dim3(NT), 0, s, p, a)
    if (p.dtype == F32) { MX4_GENERAL(F32); }
    else if (p.dtype == F16) { MX4_GENERAL(F16); }
    else { MX4_GENERAL(BF16); }
#undef MX4_GENERAL
    return hipGetLastError();
}

}  // namespace mgemm
