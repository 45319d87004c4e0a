// gs_gated_simt.cuh -- the gated projections with fp32 FMAs, for any type, size and
// alignment: 64 x 64 tiles, 4 x 4 values per thread.
#pragma once

#include "gs_gated_grad.cuh"

namespace gs {

constexpr int kSimtTile = 64, kSimtK = 16, kSimtThreads = 256;

// Stages rows r0.. and contraction steps k0.. of a matrix, element (r, k) at
// r * rs + k * ks, as fp32 at tile[k][r]; zeros outside.
template <typename T>
__device__ __forceinline__ void simt_stage(float (&tile)[kSimtK][kSimtTile + 4], const T *p,
                                           int64_t rs, int64_t ks, int64_t r0, int64_t rows, int64_t k0,
                                           int64_t K) {
#pragma unroll
    for (int i = 0; i < kSimtTile * kSimtK / kSimtThreads; ++i) {
        const int e = i * kSimtThreads + threadIdx.x;
        // neighbouring threads along the contiguous axis
        const int k = ks == 1 ? e % kSimtK : e / kSimtTile, r = ks == 1 ? e / kSimtK : e % kSimtTile;
        tile[k][r] = r0 + r < rows && k0 + k < K ? IO<T>::ld(p + (r0 + r) * rs + (k0 + k) * ks) : 0.0f;
    }
}

__device__ __forceinline__ void simt_multiply(const float (&a)[kSimtK][kSimtTile + 4],
                                              const float (&b)[kSimtK][kSimtTile + 4],
                                              float (&c)[4][4]) {
    const int tm = threadIdx.x / 16 * 4, tn = threadIdx.x % 16 * 4;
#pragma unroll
    for (int k = 0; k < kSimtK; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(&a[k][tm]);
        const float4 y = *reinterpret_cast<const float4 *>(&b[k][tn]);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) c[i][j] = fmaf(xs[i], ys[j], c[i][j]);
    }
}

template <typename T>
__global__ void __launch_bounds__(kSimtThreads) gated_simt_kernel(GatedArgs a, GatedPtrs p) {
    __shared__ __align__(16) float sx[kSimtK][kSimtTile + 4], sg[kSimtK][kSimtTile + 4],
        su[kSimtK][kSimtTile + 4];
    const int64_t tiles_n = (a.F + kSimtTile - 1) / kSimtTile;
    const int64_t m0 = blockIdx.x / tiles_n * kSimtTile, n0 = blockIdx.x % tiles_n * kSimtTile;
    float g[4][4] = {}, u[4][4] = {};
    for (int k0 = 0; k0 < a.D; k0 += kSimtK) {
        __syncthreads();
        simt_stage<T>(sx, (const T *)p.X, a.D, 1, m0, a.rows, k0, a.D);
        simt_stage<T>(sg, (const T *)p.Wg, a.D, 1, n0, a.F, k0, a.D);
        simt_stage<T>(su, (const T *)p.Wu, a.D, 1, n0, a.F, k0, a.D);
        __syncthreads();
        simt_multiply(sx, sg, g);
        simt_multiply(sx, su, u);
    }
    const int64_t m = m0 + threadIdx.x / 16 * 4, n = n0 + threadIdx.x % 16 * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (m + i >= a.rows || n + j >= a.F) continue;
            const int64_t at = (m + i) * a.F + n + j;
            float gv = g[i][j], uv = u[i][j], h = 0.0f;
            if (p.bg) {
                gv += IO<T>::ld((const T *)p.bg + n + j);
                uv += IO<T>::ld((const T *)p.bu + n + j);
            }
            with_act(a.act, [&](auto act) { h = act_of<T, decltype(act)::value>(gv) * uv; });
            ((T *)p.H)[at] = IO<T>::st(h);
            if (p.G) {
                ((T *)p.G)[at] = IO<T>::st(gv);
                ((T *)p.U)[at] = IO<T>::st(uv);
            }
        }
}

// C (M, N) = sum over segments and k of A[s](m, k) B[s](n, k), through strides.
struct SimtProduct {
    const void *A[2], *B[2];
    int64_t am, ak, bn, bk;
    int64_t M, N, K;
    int segments;
    const uint32_t *bound;   // fp16: what A is scaled by
};
template <typename T>
__global__ void __launch_bounds__(kSimtThreads) gated_simt_product_kernel(SimtProduct p, T *C) {
    __shared__ __align__(16) float sa[kSimtK][kSimtTile + 4], sb[kSimtK][kSimtTile + 4];
    const int64_t tiles_n = (p.N + kSimtTile - 1) / kSimtTile;
    const int64_t m0 = blockIdx.x / tiles_n * kSimtTile, n0 = blockIdx.x % tiles_n * kSimtTile;
    float c[4][4] = {};
    wait_for_previous_kernel(p.A[0], p.A[1]);
    for (int s = 0; s < p.segments; ++s)
        for (int64_t k0 = 0; k0 < p.K; k0 += kSimtK) {
            __syncthreads();
            simt_stage<T>(sa, (const T *)p.A[s], p.am, p.ak, m0, p.M, k0, p.K);
            simt_stage<T>(sb, (const T *)p.B[s], p.bn, p.bk, n0, p.N, k0, p.K);
            __syncthreads();
            simt_multiply(sa, sb, c);
        }
    const int64_t m = m0 + threadIdx.x / 16 * 4, n = n0 + threadIdx.x % 16 * 4;
    const float f = __is_same(T, __half) ? gated_scale(__ldg(p.bound), true) : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (m + i < p.M && n + j < p.N) C[(m + i) * p.N + n + j] = IO<T>::st(c[i][j] * f);
}

inline int64_t simt_blocks(int64_t M, int64_t N) {
    return ((M + kSimtTile - 1) / kSimtTile) * ((N + kSimtTile - 1) / kSimtTile);
}

}  // namespace gs
