// Microscaled 4-bit format (OCP Microscaling Formats MX v1.0: MXFP4) and the
// launchers of its kernels.
//
// A row of K values is cut into blocks of 32.  A block holds one scale byte b
// (E8M0: 2^(b - 127), 255 is NaN) and 32 E2M1 codes (sign, 2 exponent bits of
// bias 1, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
// to a byte with the lower k in the low nibble: 16 bytes per block.  A row is
// ceil(K / 32) blocks; codes past K in its last block are zero.
#pragma once
#include "common.h"

namespace mgemm {

constexpr int MX_BLOCK = 32;
inline int64_t mx4_blocks(int64_t K) { return (K + MX_BLOCK - 1) / MX_BLOCK; }

// Scale byte of a block whose largest magnitude has the FP32 bits `top` (the
// integer maximum of the magnitudes' bits, so a NaN or an infinity is the
// largest): floor(log2 amax) - 2, the exponent of E2M1's largest binade,
// biased by 127 and clamped to 0.  Blocks with a non-finite value get 255.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255u ? 255u : e < 2u ? 0u : e - 2u;
}
// 2^(127 - b), the factor that takes a block's values to E2M1's range
// (b <= 252 for finite blocks, so the factor is a normal number; with b = 255
// it is zero and finite values give zero codes).
__device__ __forceinline__ float mx4_factor(uint32_t b) {
    return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23);
}
// Eight codes of scaled values, lowest k in the lowest nibble.
// v_cvt_scalef32_pk_fp4_f32 with scale 1 rounds to the nearest E2M1 value,
// ties to the even mantissa; values are clamped to +-6 first.  med3 of a NaN
// gives a finite value, and the block's scale says NaN then.
__device__ __forceinline__ uint32_t mx4_pack8(const float (&x)[8], float f) {
    uint32_t w = 0;
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = __builtin_amdgcn_fmed3f(x[e] * f, -6.0f, 6.0f);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[0], t[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[2], t[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[4], t[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, t[6], t[7], 1.0f, 3);
    return w;
}
// Value of a code (its low four bits), before the block's scale.
__device__ __forceinline__ float mx4_value(uint32_t c) {
    const uint32_t m = c & 7u;
    const float v = m < 2u ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
    return (c & 8u) ? -v : v;
}
// v times 2^(b - 127), NaN for b = 255.
__device__ __forceinline__ float mx4_scaled(float v, uint32_t b) {
    return b == 255u ? __uint_as_float(0x7FC00000u) : __builtin_amdgcn_ldexpf(v, (int)b - 127);
}

// Eight elements at x + 16 B (16-bit) or 32 B (FP32) apart, as FP32.
template <int XT>
__device__ __forceinline__ void load8(const void* x, float (&v)[8]) {
    if constexpr (XT == F32) {
        const f32x4 a = *(const f32x4*)x, b = *((const f32x4*)x + 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    } else {
        const u32x4 w = *(const u32x4*)x;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = from_bits<XT>((uint16_t)(w[e / 2] >> (16 * (e & 1))));
    }
}
template <int XT>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
    return Elem<XT>::load((const typename Elem<XT>::T*)x, i);
}

// Stores up to four outputs of one row from v = alpha * acc: adds beta * C,
// rounds once.  n + e < lim selects the outputs that exist.
template <int CT>
__device__ __forceinline__ void mx4_store4(void* C, int64_t row, int n, int lim, bool vec_ok, float beta,
                                           float (&v)[4]) {
    if constexpr (CT == F32) {
        float* c = (float*)C + row;
        if (beta != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < lim) v[e] = fmaf(beta, c[n + e], v[e]);
        }
        if (vec_ok && n + 4 <= lim) {
            *(f32x4*)(c + n) = f32x4{v[0], v[1], v[2], v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < lim) c[n + e] = v[e];
        }
    } else {
        store_out4<CT, EPI_NONE>((uint16_t*)C + row, n, lim, vec_ok, beta, v);
    }
}
// Whether four consecutive outputs of a row may be stored as one vector.
template <int CT>
__device__ __forceinline__ bool mx4_vec_ok(const void* C, int64_t ldc) {
    constexpr int B = CT == F32 ? 16 : 8;
    return ldc % 4 == 0 && ((uintptr_t)C & (B - 1)) == 0;
}

// Operands of a product beyond the Problem: p.A and p.B hold codes (byte
// strides p.lda and p.ldb), p.B2 the codes of the gated pair's second matrix.
struct Mx4Args {
    const uint8_t* sa;    // scale rows of A, byte stride ldsa
    int64_t ldsa;
    const uint8_t* sb;    // scale rows of B (and of B2: sb2), byte stride ldsb
    const uint8_t* sb2;
    int64_t ldsb;
    float* part;          // split K: [tile][range][chunk][thread] f32x4 partial sums
    int ksplit;           // K ranges (1: no split)
    int nks;              // 128-element slices per range (the last may hold fewer)
    const void* X;        // decode kernel only: activations to quantise in the kernel
    int64_t ldx;          //   (16-bit or FP32 elements of type xtype), or null for codes in p.A
    int xtype;
};

hipError_t launch_quantize_mx4(int64_t M, int64_t K, const void* X, int64_t ldx, int xtype, uint8_t* Q,
                               int64_t ldq, uint8_t* S, int64_t lds, hipStream_t s);
hipError_t launch_dequantize_mx4(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                                 int64_t lds, void* Y, int64_t ldy, int ytype, hipStream_t s);
// Any alignment: scalar products of decoded codes.
hipError_t launch_mx4_general(const Problem& p, const Mx4Args& a, hipStream_t s);
// MFMA tiles of bm x bn (256x256, 256x192, 128x192, 64x192; the gated pair:
// 192 wide, 96 columns of each matrix).
bool mx4_mfma_supports(const Problem& p, const Mx4Args& a, int bn, int bm);
int mx4_splits(const Problem& p, int bn, int bm, int requested, const Workspace& ws);
hipError_t launch_mx4_mfma(const Problem& p, Mx4Args a, int bn, int bm, int ksplit, const Workspace& ws,
                           hipStream_t s);
// Decode shapes: M <= 64 (M <= 16 when the activations are quantised in the kernel).
bool mx4_skinny_supports(const Problem& p, const Mx4Args& a);
hipError_t launch_mx4_skinny(const Problem& p, const Mx4Args& a, hipStream_t s);

}  // namespace mgemm
