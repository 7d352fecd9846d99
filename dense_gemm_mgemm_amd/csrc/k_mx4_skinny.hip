// Microscaled 4-bit products for few rows (M <= 64): a stream of the weights.
//
// A workgroup of eight waves owns 16 * NTW output columns and all of K; wave
// w takes the steps w, w + 8, ... of one or two adjacent 128-element slices (a
// 128-byte line) of every row, and the waves' FP32 sums are added in wave order
// through LDS: the result does not depend on timing and there is no second
// launch.  Weights go from memory to registers: lane l of
// v_mfma_scale_f32_16x16x128_f8f6f4 holds block l/16 of row l%16, which is one
// 16-byte load, and its scale is one byte of the slice's dword of four.  The
// next step's slices are requested before the present ones are multiplied.
//
// Bound by the weights' bytes and the launch: 1 / 4 / 16 x 12288 x 4096 from codes
// 8.6 to 8.9 / 9.0 to 9.5 / 10.4 to 10.9 us (26.7 MB: 5.5 at a copy's rate), with the
// quantisation 10.6 to 11.1 / 10.6 to 10.8 / 12.6 to 13.2; the gated pair of 4 rows
// 16.6 to 17.2 (53 MB).  With the quantisation of up to 4 rows, the pair and two
// column tiles hold 139 to 141 registers (16-bit X), so a CU has room for one
// workgroup and not two, and 384 or 768 of them end in a round that is half empty;
// from codes they hold 123.
//
// Few short rows are quantised here (RM rows at most, as 16-byte loads of
// eight elements, four lanes to a block), each wave for its own slices through
// a private piece of LDS, which saves a launch and the round trip of the codes;
// the work grows with M and K and is repeated by every workgroup.  Others read
// codes made by k_mx4_quant.
#include "mx4.h"

namespace mgemm {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int NW = 8, NT = 64 * NW;
constexpr int LROW = 80;                 // LDS bytes per quantised 64-byte row: 16 rows hit 16 different bank groups

// Orders LDS accesses between the lanes of one wave: the hardware keeps a
// wave's LDS operations in order, so only the compiler has to be told.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ f32x4 mfma4(i32x4 x, i32x4 y, f32x4 c, int sx, int sy) {
    const i32x8 xa = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8 ya = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(xa, ya, c, 4, 4, 0, sx, 0, sy);
}

// XT >= 0: activations of that type, at most RM rows, quantised here; XT < 0:
// codes, MT blocks of 16 rows.  NB: 1, or 2 for the gated pair.
template <int CT, int XT, int RM, int MT, int NTW, int NB>
__global__ __launch_bounds__(NT) void k_mx4_skinny(Problem p, Mx4Args f) {
    constexpr bool QX = XT >= 0;
    static_assert(!QX || MT == 1, "quantised in the kernel: one block of rows");
    constexpr int U = QX && RM == 16 ? 1 : 2;             // slices of a wave per step
    constexpr int TILES = NTW * NB * MT;
    static_assert(TILES <= 8, "the sum over waves takes one wave per tile");
    constexpr int CL = QX ? U * RM / 4 : 1;               // eight-element chunks per lane and step
    constexpr int XS = XT == F32 ? 4 : 2;
    constexpr int QBYTES = QX ? NW * U * 16 * (LROW + 4) : 0, RBYTES = NW * TILES * 64 * 16;
    __shared__ __align__(16) unsigned char smem[QBYTES > RBYTES ? QBYTES : RBYTES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NTW);
    const int blocks = (int)((p.K + MX_BLOCK - 1) / MX_BLOCK);
    const int steps = (blocks + 4 * U - 1) / (4 * U);     // U adjacent slices each
    const int lr = lane & 15, lc = lane >> 4;             // this lane's row of a tile and block of a slice

    const uint8_t* w[NTW * NB];
    const uint8_t* ws[NTW * NB];
#pragma unroll
    for (int t = 0; t < NTW * NB; ++t) {
        int64_t n = n0 + 16 * (t / NB) + lr;
        n = n < p.N ? n : p.N - 1;
        w[t] = (const uint8_t*)(t % NB ? p.B2 : p.B) + n * p.ldb + 16 * lc;
        ws[t] = (t % NB ? f.sb2 : f.sb) + n * f.ldsb;
    }
    const uint8_t* a[MT];
    const uint8_t* as[MT];
    if constexpr (!QX) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            int64_t m = 16 * t + lr;
            m = m < p.M ? m : p.M - 1;
            a[t] = (const uint8_t*)p.A + m * p.lda + 16 * lc;
            as[t] = f.sa + m * f.ldsa;
        }
    }
    typedef unsigned Sc __attribute__((ext_vector_type(U)));
    struct Step {
        u32x4 x[CL][XT == F32 ? 2 : 1];
        i32x4 w[U][NTW * NB];
        int ws[U][NTW * NB];
        i32x4 a[U][QX ? 1 : MT];
        int as[U][QX ? 1 : MT];
    };
    // Requests step q: the activations first (they come from L2, are waited for
    // first and are quantised while the weights are still on their way), then
    // a row's codes and the scales of its U slices in one load.  Blocks past K
    // read as zero codes with scale 1.
    auto request = [&](Step& st, int q) {
        if constexpr (QX) {
            // Chunk c = 64 i + lane of the step: slice c / (16 RM), row
            // (c / 16) % RM, elements 8 (c % 16) of the slice.
#pragma unroll
            for (int i = 0; i < CL; ++i) {
                const int c = 64 * i + lane, m = (c >> 4) % RM;
                const int64_t k = (int64_t)(U * q + c / (16 * RM)) * 128 + 8 * (c & 15);
                const unsigned char* x = (const unsigned char*)f.X + (m * f.ldx + k) * XS;
                u32x4 v[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
                if (m < p.M && k + 8 <= p.K) {
                    v[0] = *(const u32x4*)x;
                    if constexpr (XT == F32) v[1] = *((const u32x4*)x + 1);
                } else if (m < p.M && k < p.K) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (k + e >= p.K) break;
                        if constexpr (XT == F32) v[e / 4][e % 4] = ((const uint32_t*)x)[e];
                        else v[0][e / 2] |= (uint32_t)((const uint16_t*)x)[e] << (16 * (e % 2));
                    }
                }
                st.x[i][0] = v[0];
                if constexpr (XT == F32) st.x[i][1] = v[1];
            }
        }
        auto row = [&](const uint8_t* codes, const uint8_t* scales, i32x4* c0, int* s0, int stride) {
            Sc sc;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = 4 * (U * q + u) + lc < blocks;
                c0[u * stride] = in ? *(const i32x4*)(codes + (int64_t)(U * q + u) * 64) : i32x4{0, 0, 0, 0};
            }
            sc = q < steps ? *(const Sc*)(scales + (int64_t)q * (4 * U)) : Sc{};
#pragma unroll
            for (int u = 0; u < U; ++u)
                s0[u * stride] = 4 * (U * q + u) + lc < blocks ? (int)(sc[u] >> (8 * lc)) : 127;
        };
#pragma unroll
        for (int t = 0; t < NTW * NB; ++t) row(w[t], ws[t], &st.w[0][t], &st.ws[0][t], NTW * NB);
        if constexpr (!QX) {
#pragma unroll
            for (int t = 0; t < MT; ++t) row(a[t], as[t], &st.a[0][t], &st.as[0][t], MT);
        }
    };

    unsigned char* qx = smem + wave * (U * 16 * (LROW + 4));      // this wave's codes, then its scales
    unsigned char* qs = qx + U * 16 * LROW;
    if constexpr (QX) {
        // Rows past M stay zero codes with scale 1.
        for (int i = lane; i < U * 16 * LROW / 4; i += 64) ((uint32_t*)qx)[i] = 0;
        if (lane < U * 16) ((uint32_t*)qs)[lane] = 0x7F7F7F7Fu;
    }
    auto quantise = [&](const Step& st) {
#pragma unroll
        for (int i = 0; i < CL; ++i) {
            const int c = 64 * i + lane, u = c / (16 * RM), m = (c >> 4) % RM, part = c & 15;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (XT == F32) v[e] = __uint_as_float(st.x[i][e / 4][e % 4]);
                else v[e] = from_bits<XT>((uint16_t)(st.x[i][0][e / 2] >> (16 * (e % 2))));
            }
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                top = b > top ? b : top;
            }
            uint32_t o = (uint32_t)__shfl_xor((int)top, 1, 64);
            top = o > top ? o : top;
            o = (uint32_t)__shfl_xor((int)top, 2, 64);
            top = o > top ? o : top;
            const uint32_t b = mx4_scale_byte(top);
            uint32_t q = mx4_pack8(v, mx4_factor(b));
            if (b == 255u) q = 0;
            *(uint32_t*)(qx + (u * 16 + m) * LROW + 4 * part) = q;
            if ((part & 3) == 0) qs[(u * 16 + m) * 4 + (part >> 2)] = (uint8_t)b;
        }
    };

    f32x4 acc[NTW * NB][MT];
#pragma unroll
    for (int t = 0; t < NTW * NB; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto multiply = [&](const Step& st) {
        if constexpr (QX) {
            wave_fence();
            quantise(st);
            wave_fence();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                i32x4 xa;
                int xs;
                if constexpr (QX) {
                    xa = *(const i32x4*)(qx + (u * 16 + lr) * LROW + 16 * lc);
                    xs = qs[(u * 16 + lr) * 4 + lc];
                } else {
                    xa = st.a[u][m];
                    xs = st.as[u][m];
                }
#pragma unroll
                for (int t = 0; t < NTW * NB; ++t) acc[t][m] = mfma4(st.w[u][t], xa, acc[t][m], st.ws[u][t], xs);
            }
    };

    Step s0, s1;
    request(s0, wave);
    for (int q = wave; q < steps; q += 2 * NW) {
        request(s1, q + NW);
        multiply(s0);
        request(s0, q + 2 * NW);
        multiply(s1);
    }

    // Sum over the waves in wave order: wave t adds tile t.
    __syncthreads();
    f32x4* part = (f32x4*)smem;
#pragma unroll
    for (int t = 0; t < NTW * NB; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[(wave * TILES + t * MT + m) * 64 + lane] = acc[t][m];
    __syncthreads();
    auto sum = [&](int tile) {
        f32x4 v = part[tile * 64 + lane];
#pragma unroll
        for (int i = 1; i < NW; ++i) v = v + part[(i * TILES + tile) * 64 + lane];
        return v;
    };
    if (wave >= NTW * MT) return;
    const int t = wave / MT, mt = wave % MT;              // column tile and row block
    const f32x4 g = sum(t * NB * MT + mt);
    float v[4];
    if constexpr (NB == 2) {
        const f32x4 u = sum((t * NB + 1) * MT + mt);
        gated_product4<CT>({g[0], g[1], g[2], g[3]}, {u[0], u[1], u[2], u[3]}, v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = p.alpha * g[e];
    }
    const int64_t m = 16 * mt + lr;
    if (m >= p.M) return;
    const int64_t left = p.N - n0;
    mx4_store4<CT>(p.C, m * p.ldc + n0, 16 * t + 4 * lc, (int)(left < 16 * NTW ? left : 16 * NTW),
                   mx4_vec_ok<CT>(p.C, p.ldc), p.beta, v);
}

template <int CT, int XT, int RM, int MT, int NTW, int NB>
hipError_t go(const Problem& p, const Mx4Args& a, hipStream_t s) {
    hipLaunchKernelGGL((k_mx4_skinny<CT, XT, RM, MT, NTW, NB>), dim3((unsigned)((p.N + 16 * NTW - 1) / (16 * NTW))),
                       dim3(NT), 0, s, p, a);
    return hipGetLastError();
}

// One column tile per wave for the gated pair and for N whose tiles would
// otherwise leave CUs without a workgroup; two elsewhere.
template <int CT, int XT, int RM, int MT>
hipError_t by_width(const Problem& p, const Mx4Args& a, hipStream_t s) {
    if (p.B2 != nullptr) return go<CT, XT, RM, MT, 1, 2>(p, a, s);
    const int64_t cu = p.num_cu > 0 ? p.num_cu : 256;
    if (p.N <= 32 * cu) return go<CT, XT, RM, MT, 1, 1>(p, a, s);
    return go<CT, XT, RM, MT, 2, 1>(p, a, s);
}

template <int CT>
hipError_t by_rows(const Problem& p, const Mx4Args& a, hipStream_t s) {
    if (a.X != nullptr) {
#define MX4_X(XT)                                                 \
    case XT:                                                      \
        return p.M <= 4 ? by_width<CT, XT, 4, 1>(p, a, s) : by_width<CT, XT, 16, 1>(p, a, s)
        switch (a.xtype) {
        MX4_X(F32);
        MX4_X(F16);
        default:
        MX4_X(BF16);
        }
#undef MX4_X
    }
    if (p.M <= 16) return by_width<CT, -1, 16, 1>(p, a, s);
    if (p.M <= 32) return by_width<CT, -1, 16, 2>(p, a, s);
    return by_width<CT, -1, 16, 4>(p, a, s);
}

}  // namespace

bool mx4_skinny_supports(const Problem& p, const Mx4Args& a) {
    auto al = [](const void* q) { return ((uintptr_t)q & 15) == 0; };
    if (p.M > (a.X != nullptr ? 16 : 64)) return false;
    if (p.ldb % 16 != 0 || !al(p.B) || !al(p.B2)) return false;
    // A step's scales are one load of up to eight bytes.
    auto al8 = [](const void* q) { return ((uintptr_t)q & 7) == 0; };
    if (a.ldsb % 8 != 0 || !al8(a.sb) || !al8(a.sb2)) return false;
    if (a.X == nullptr && (a.ldsa % 8 != 0 || !al8(a.sa))) return false;
    if (a.X != nullptr) {
        const int es = a.xtype == F32 ? 4 : 2;
        if (a.ldx * es % 16 != 0 || !al(a.X)) return false;
    } else if (p.lda % 16 != 0 || !al(p.A)) {
        return false;
    }
    return mx4_blocks(p.K) <= 0x3fffffff && (p.N + 15) / 16 <= 0x7fffffff;
}

hipError_t launch_mx4_skinny(const Problem& p, const Mx4Args& a, hipStream_t s) {
    if (p.dtype == F32) return by_rows<F32>(p, a, s);
    if (p.dtype == F16) return by_rows<F16>(p, a, s);
    return by_rows<BF16>(p, a, s);
}

}  // namespace mgemm
