// Microscaled 4-bit quantisation (values -> codes and scales) and its inverse.
//
// Four lanes share a block of 32: each holds eight consecutive elements (one
// 16-byte load of a 16-bit type, two of FP32), the block's largest magnitude
// is an integer maximum over the four lanes, and each lane converts and
// stores four bytes of codes.  Work is one flat sequence of eight-element
// chunks over all rows, so short rows fill waves too.
//
// Bound by memory: 12288 x 4096 FP32 quantised in 35 to 55 us and read back in 39 to
// 41 (201 MB of values each way).  16 x 4096 BF16: 2.3 and 2.5 us, launches.
#include "mx4.h"

namespace mgemm {
namespace {

constexpr int NT = 256;
// Chunks per thread, all loaded before the first is used: R_LARGE where that
// leaves every CU two workgroups (12288 x 4096 FP32 quantised and read back
// 96 us, 4.5 TB/s), one elsewhere (latency).
constexpr int R_LARGE = 4, FILL = 512;

// VEC: X rows are 16-byte aligned and Q rows 4-byte aligned.  total = M *
// per_row chunks, at most 2^31 (the launcher cuts taller matrices).
template <int XT, bool VEC, int R>
__global__ __launch_bounds__(NT) void k_mx4_quant(uint32_t total, uint32_t per_row, int64_t K, const void* X,
                                                  int64_t ldx, uint8_t* Q, int64_t ldq, uint8_t* S,
                                                  int64_t lds) {
    constexpr int ES = XT == F32 ? 4 : 2;
    float v[R][8];
    uint32_t row[R], chunk[R];
    const uint32_t first = blockIdx.x * (NT * R) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t t = first + i * NT;
        row[i] = t / per_row;
        chunk[i] = t - row[i] * per_row;
        const int64_t k = (int64_t)chunk[i] * 8;
        const unsigned char* x = (const unsigned char*)X + ((int64_t)row[i] * ldx + k) * ES;
        if (VEC && t < total && k + 8 <= K) {
            load8<XT>(x, v[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = t < total && k + e < K ? load1<XT>(x, e) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t b = __float_as_uint(v[i][e]) & 0x7FFFFFFFu;
            top = b > top ? b : top;
        }
        // per_row is a multiple of 4 and NT * R of 64, so a block's four
        // lanes are always one aligned group of four.
        uint32_t o = (uint32_t)__shfl_xor((int)top, 1, 64);
        top = o > top ? o : top;
        o = (uint32_t)__shfl_xor((int)top, 2, 64);
        top = o > top ? o : top;
        if (first + i * NT >= total) continue;
        const uint32_t b = mx4_scale_byte(top);
        uint32_t w = mx4_pack8(v[i], mx4_factor(b));
        if (b == 255u) w = 0;
        uint8_t* q = Q + (int64_t)row[i] * ldq + (int64_t)chunk[i] * 4;
        if (VEC) {
            *(uint32_t*)q = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) q[e] = (uint8_t)(w >> (8 * e));
        }
        if ((chunk[i] & 3u) == 0) S[(int64_t)row[i] * lds + (chunk[i] >> 2)] = (uint8_t)b;
    }
}

template <int YT, bool VEC, int R>
__global__ __launch_bounds__(NT) void k_mx4_dequant(uint32_t total, uint32_t per_row, int64_t K,
                                                    const uint8_t* Q, int64_t ldq, const uint8_t* S,
                                                    int64_t lds, void* Y, int64_t ldy) {
    uint32_t w[R], b[R], row[R], chunk[R];
    const uint32_t first = blockIdx.x * (NT * R) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t t = first + i * NT;
        row[i] = t / per_row;
        chunk[i] = t - row[i] * per_row;
        w[i] = b[i] = 0;
        if (t >= total) continue;
        const uint8_t* q = Q + (int64_t)row[i] * ldq + (int64_t)chunk[i] * 4;
        if (VEC) {
            w[i] = *(const uint32_t*)q;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[i] |= (uint32_t)q[e] << (8 * e);
        }
        b[i] = S[(int64_t)row[i] * lds + (chunk[i] >> 2)];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (first + i * NT >= total) continue;
        const int64_t k = (int64_t)chunk[i] * 8;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = mx4_scaled(mx4_value(w[i] >> (4 * e)), b[i]);
        using T = typename Elem<YT>::T;
        T* y = (T*)Y + (int64_t)row[i] * ldy + k;
        if (VEC && k + 8 <= K) {
            if constexpr (YT == F32) {
                *(f32x4*)y = f32x4{v[0], v[1], v[2], v[3]};
                *((f32x4*)y + 1) = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                u32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[e] = (uint32_t)to_bits<YT>(v[2 * e]) | ((uint32_t)to_bits<YT>(v[2 * e + 1]) << 16);
                *(u32x4*)y = o;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < K) Elem<YT>::store(y, e, v[e]);
        }
    }
}

// Rows are cut into launches of at most 2^31 chunks (32-bit indices; the row
// pointers are 64-bit).  Rows longer than that are refused by the caller.
template <class F>
hipError_t by_rows(int64_t M, int64_t K, F&& launch) {
    const int64_t per_row = mx4_blocks(K) * 4;
    const int64_t step = ((int64_t)1 << 31) / per_row;
    for (int64_t m = 0; m < M; m += step) {
        const int64_t rows = M - m < step ? M - m : step;
        const uint32_t total = (uint32_t)(rows * per_row);
        const bool large = total >= (uint32_t)NT * R_LARGE * FILL;
        const uint32_t per_wg = NT * (large ? R_LARGE : 1);
        launch(m, total, (uint32_t)per_row, dim3((unsigned)(((uint64_t)total + per_wg - 1) / per_wg)), large);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int XT>
hipError_t quant(int64_t M, int64_t K, const void* X, int64_t ldx, uint8_t* Q, int64_t ldq, uint8_t* S,
                 int64_t lds, hipStream_t s) {
    constexpr int ES = XT == F32 ? 4 : 2;
    const bool vec = ldx * ES % 16 == 0 && ((uintptr_t)X & 15) == 0 && ldq % 4 == 0 && ((uintptr_t)Q & 3) == 0;
    return by_rows(M, K, [&](int64_t m, uint32_t total, uint32_t per_row, dim3 grid, bool large) {
        const void* x = (const unsigned char*)X + m * ldx * ES;
        auto kern = vec ? (large ? k_mx4_quant<XT, true, R_LARGE> : k_mx4_quant<XT, true, 1>)
                        : (large ? k_mx4_quant<XT, false, R_LARGE> : k_mx4_quant<XT, false, 1>);
        hipLaunchKernelGGL(kern, grid, dim3(NT), 0, s, total, per_row, K, x, ldx, Q + m * ldq, ldq, S + m * lds, lds);
    });
}

template <int YT>
hipError_t dequant(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* S, int64_t lds, void* Y,
                   int64_t ldy, hipStream_t s) {
    constexpr int ES = YT == F32 ? 4 : 2;
    const bool vec = ldy * ES % 16 == 0 && ((uintptr_t)Y & 15) == 0 && ldq % 4 == 0 && ((uintptr_t)Q & 3) == 0;
    return by_rows(M, K, [&](int64_t m, uint32_t total, uint32_t per_row, dim3 grid, bool large) {
        void* y = (unsigned char*)Y + m * ldy * ES;
        auto kern = vec ? (large ? k_mx4_dequant<YT, true, R_LARGE> : k_mx4_dequant<YT, true, 1>)
                        : (large ? k_mx4_dequant<YT, false, R_LARGE> : k_mx4_dequant<YT, false, 1>);
        hipLaunchKernelGGL(kern, grid, dim3(NT), 0, s, total, per_row, K, Q + m * ldq, ldq, S + m * lds, lds, y, ldy);
    });
}

}  // namespace

hipError_t launch_quantize_mx4(int64_t M, int64_t K, const void* X, int64_t ldx, int xtype, uint8_t* Q,
                               int64_t ldq, uint8_t* S, int64_t lds, hipStream_t s) {
    if (xtype == F32) return quant<F32>(M, K, X, ldx, Q, ldq, S, lds, s);
    if (xtype == F16) return quant<F16>(M, K, X, ldx, Q, ldq, S, lds, s);
    return quant<BF16>(M, K, X, ldx, Q, ldq, S, lds, s);
}

hipError_t launch_dequantize_mx4(int64_t M, int64_t K, const uint8_t* Q, int64_t ldq, const uint8_t* S,
                                 int64_t lds, void* Y, int64_t ldy, int ytype, hipStream_t s) {
    if (ytype == F32) return dequant<F32>(M, K, Q, ldq, S, lds, Y, ldy, s);
    if (ytype == F16) return dequant<F16>(M, K, Q, ldq, S, lds, Y, ldy, s);
    return dequant<BF16>(M, K, Q, ldq, S, lds, Y, ldy, s);
}

}  // namespace mgemm
