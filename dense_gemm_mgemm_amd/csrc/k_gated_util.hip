// Elementwise kernels of the gated block: dG and dU from stored G and U, and
// the copy of operands that the matrix kernels cannot read in place.  Both are
// bound by memory: eight elements a thread, 16-byte accesses where rows allow
// (dG and dU of 1024 x 12288 BF16: 126 MB in 27 us, 4.7 TB/s; a 4 GiB copy
// reaches 4.84).
#include "gated_tile.h"

namespace mgemm {
namespace {

template <int DT>
__device__ __forceinline__ void load8(const uint16_t* p, int64_t left, bool vec, float (&v)[8]) {
    if (vec && left >= 8) {
        const u32x4 w = *(const u32x4*)p;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = from_bits<DT>((uint16_t)(w[e / 2] >> (16 * (e & 1))));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < left ? from_bits<DT>(p[e]) : 0.0f;
    }
}
template <int DT>
__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = (uint32_t)to_bits<DT>(v[2 * e]) | ((uint32_t)to_bits<DT>(v[2 * e + 1]) << 16);
    *(u32x4*)p = w;
}

// Rows of per_row chunks of eight, zeros past M x N.
template <int DT>
__global__ __launch_bounds__(NT) void k_gated_grad(uint32_t total, uint32_t per_row, int64_t M, int64_t N,
                                                   const uint16_t* G,
                                                   const uint16_t* U, int64_t ldg, const uint16_t* dZ, int64_t lddz,
                                                   uint16_t* dG, uint16_t* dU, int64_t ldd, bool vec) {
    const uint32_t t = blockIdx.x * NT + threadIdx.x;
    if (t >= total) return;
    const uint32_t row = t / per_row;
    const int64_t n = (int64_t)(t - row * per_row) * 8;
    float g[8], u[8], dz[8], a[8], b[8];
    const int64_t left = row < M ? N - n : 0;
    load8<DT>(G + row * ldg + n, left, vec, g);
    load8<DT>(U + row * ldg + n, left, vec, u);
    load8<DT>(dZ + row * lddz + n, left, vec, dz);
    gated_grad(g, u, dz, a, b);
    store8<DT>(dG + row * ldd + n, a);
    store8<DT>(dU + row * ldd + n, b);
}

// A row's eight elements at any 2-byte alignment (the hardware's unaligned
// loads; memcpy lets the compiler choose them).
__global__ __launch_bounds__(NT) void k_repack(Repack r) {
    const int i = blockIdx.y;
    const uint32_t per_row = (uint32_t)(r.ldd[i] / 8);
    const int64_t total = r.rows_out[i] * per_row;
    const uint16_t* src = (const uint16_t*)r.src[i];
    uint16_t* dst = (uint16_t*)r.dst[i];
    for (int64_t t = (int64_t)blockIdx.x * NT + threadIdx.x; t < total; t += (int64_t)gridDim.x * NT) {
        const int64_t row = total <= 0xffffffffu ? (int64_t)((uint32_t)t / per_row) : t / per_row;
        const int64_t c = (t - row * per_row) * 8;
        const uint16_t* s = src + row * r.lds[i] + c;
        const int64_t left = row < r.rows[i] ? r.cols[i] - c : 0;
        u32x4 v = u32x4{0, 0, 0, 0};
        if (left >= 8) {
            __builtin_memcpy(&v, s, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < left) v[e / 2] |= (uint32_t)s[e] << (16 * (e & 1));
        }
        *(u32x4*)(dst + row * r.ldd[i] + c) = v;
    }
}

}  // namespace

hipError_t launch_gated_grad(int64_t M, int64_t N, int64_t Mo, int64_t No, const void* G, const void* U, int64_t ldg,
                             const void* dZ, int64_t lddz, void* dG, void* dU, int64_t ldd, int dtype,
                             hipStream_t s) {
    const int64_t per_row = No / 8, step = ((int64_t)1 << 31) / per_row;
    auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
    const bool vec = ldg % 8 == 0 && lddz % 8 == 0 && al(G) && al(U) && al(dZ);
    for (int64_t m = 0; m < Mo; m += step) {
        const int64_t rows = Mo - m < step ? Mo - m : step;
        const uint32_t total = (uint32_t)(rows * per_row);
        auto kern = dtype == F16 ? k_gated_grad<F16> : k_gated_grad<BF16>;
        hipLaunchKernelGGL(kern, dim3((total + NT - 1) / NT), dim3(NT), 0, s, total, (uint32_t)per_row, M - m, N,
                           (const uint16_t*)G + m * ldg, (const uint16_t*)U + m * ldg, ldg,
                           (const uint16_t*)dZ + m * lddz, lddz, (uint16_t*)dG + m * ldd, (uint16_t*)dU + m * ldd,
                           ldd, vec);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_repack(const Repack& r, hipStream_t s) {
    int64_t most = 0;
    for (int i = 0; i < r.n; ++i) {
        const int64_t c = r.rows_out[i] * (r.ldd[i] / 8);
        most = c > most ? c : most;
    }
    if (most == 0) return hipSuccess;
    const int64_t blocks = (most + NT - 1) / NT;
    hipLaunchKernelGGL(k_repack, dim3((unsigned)(blocks < 4096 ? blocks : 4096), (unsigned)r.n), dim3(NT), 0, s, r);
    return hipGetLastError();
}

}  // namespace mgemm
