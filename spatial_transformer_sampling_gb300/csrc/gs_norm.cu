// gs_norm.cu -- layer norm over the last axis, forward and backward.
//
// Forward, per row x of D elements (fp32 throughout, one rounding at the store):
//   mean = sum x / D, var = sum (x - mean)^2 / D, inv = 1 / sqrt(var + eps),
//   y = (x - mean) * inv * scale + B.
// Backward, with xhat = (x - mean) * inv and g = dy * scale:
//   dx = inv * (g - sum(g) / D - xhat * sum(g * xhat) / D),
//   dscale = sum over rows of dy * xhat,  dB = sum over rows of dy.
#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One warp per row.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_kernel(const T *X, const T *scale, const T *B, T *Y, float *mean, float *inv,
                      NormArgs a) {
    const int64_t row = (int64_t)blockIdx.x * (kNormThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= a.rows) return;
    const T *x = X + row * a.D;
    float s = 0.0f;
    for (int i = lane; i < a.D; i += 32) s += IO<T>::ld(x + i);
    const float m = warp_sum(s) / (float)a.D;
    float v = 0.0f;
    for (int i = lane; i < a.D; i += 32) {
        const float d = IO<T>::ld(x + i) - m;
        v = fmaf(d, d, v);
    }
    const float r = 1.0f / sqrtf(warp_sum(v) / (float)a.D + a.eps);
    for (int i = lane; i < a.D; i += 32) {
        const float b = B ? IO<T>::ld(B + i) : 0.0f;
        Y[row * a.D + i] = IO<T>::st(fmaf((IO<T>::ld(x + i) - m) * r, IO<T>::ld(scale + i), b));
    }
    if (lane == 0) {
        if (mean) mean[row] = m;
        if (inv) inv[row] = r;
    }
}

template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_dx_kernel(const T *dY, const T *X, const T *scale, const float *mean,
                         const float *inv, T *dX, NormArgs a) {
    const int64_t row = (int64_t)blockIdx.x * (kNormThreads / 32) + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (row >= a.rows) return;
    const T *x = X + row * a.D, *dy = dY + row * a.D;
    const float m = mean[row], r = inv[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int i = lane; i < a.D; i += 32) {
        const float g = IO<T>::ld(dy + i) * IO<T>::ld(scale + i);
        s0 += g;
        s1 = fmaf(g, (IO<T>::ld(x + i) - m) * r, s1);
    }
    s0 = warp_sum(s0) / (float)a.D;
    s1 = warp_sum(s1) / (float)a.D;
    for (int i = lane; i < a.D; i += 32) {
        const float g = IO<T>::ld(dy + i) * IO<T>::ld(scale + i);
        const float xh = (IO<T>::ld(x + i) - m) * r;
        dX[row * a.D + i] = IO<T>::st(r * (g - s0 - xh * s1));
    }
}

// Column sums of one block of rows: a thread per column, rows in order.
template <typename T>
__global__ void layer_norm_partial_kernel(const T *dY, const T *X, const float *mean,
                                          const float *inv, float *partials, int64_t rows_per,
                                          NormArgs a) {
    const int col = blockIdx.x * blockDim.x + threadIdx.x;
    if (col >= a.D) return;
    const int64_t r0 = blockIdx.y * rows_per, r1 = min(r0 + rows_per, a.rows);
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t row = r0; row < r1; ++row) {
        const float dy = IO<T>::ld(dY + row * a.D + col);
        s0 = fmaf(dy, (IO<T>::ld(X + row * a.D + col) - mean[row]) * inv[row], s0);
        s1 += dy;
    }
    partials[((int64_t)blockIdx.y * 2) * a.D + col] = s0;
    partials[((int64_t)blockIdx.y * 2 + 1) * a.D + col] = s1;
}

template <typename T>
__global__ void layer_norm_finish_kernel(const float *partials, int blocks, T *dScale, T *dB,
                                         int D) {
    const int col = blockIdx.x * blockDim.x + threadIdx.x;
    if (col >= D) return;
    float s0 = 0.0f, s1 = 0.0f;
    for (int b = 0; b < blocks; ++b) {
        s0 += partials[((int64_t)b * 2) * D + col];
        s1 += partials[((int64_t)b * 2 + 1) * D + col];
    }
    if (dScale) dScale[col] = IO<T>::st(s0);
    if (dB) dB[col] = IO<T>::st(s1);
}

}  // namespace

int layer_norm_partial_blocks(int64_t rows, int64_t D) {
    (void)D;
    const int64_t b = (rows + 63) / 64;
    return (int)(b < 1 ? 1 : b > 608 ? 608 : b);
}

template <typename T>
cudaError_t launch_layer_norm(const void *X, const void *scale, const void *B, void *Y, float *mean,
                              float *inv, const NormArgs &a, cudaStream_t s) {
    const int64_t blocks = (a.rows + kNormThreads / 32 - 1) / (kNormThreads / 32);
    layer_norm_kernel<T><<<(unsigned)blocks, kNormThreads, 0, s>>>(
        (const T *)X, (const T *)scale, (const T *)B, (T *)Y, mean, inv, a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_layer_norm_backward(const void *dY, const void *X, const void *scale,
                                       const float *mean, const float *inv, void *dX, void *dScale,
                                       void *dB, float *partials, const NormArgs &a,
                                       cudaStream_t s) {
    if (a.rows > 0) {
        const int64_t blocks = (a.rows + kNormThreads / 32 - 1) / (kNormThreads / 32);
        layer_norm_dx_kernel<T><<<(unsigned)blocks, kNormThreads, 0, s>>>(
            (const T *)dY, (const T *)X, (const T *)scale, mean, inv, (T *)dX, a);
    }
    if (dScale || dB) {
        const int nb = a.rows > 0 ? layer_norm_partial_blocks(a.rows, a.D) : 0;
        const unsigned cols = (unsigned)((a.D + 127) / 128);
        if (nb > 0)
            layer_norm_partial_kernel<T><<<dim3(cols, nb), 128, 0, s>>>(
                (const T *)dY, (const T *)X, mean, inv, partials, (a.rows + nb - 1) / nb, a);
        layer_norm_finish_kernel<T><<<cols, 128, 0, s>>>(partials, nb, (T *)dScale, (T *)dB, a.D);
    }
    return cudaGetLastError();
}

#define GS_NORM_INST(T)                                                                           \
    template cudaError_t launch_layer_norm<T>(const void *, const void *, const void *, void *,   \
                                              float *, float *, const NormArgs &, cudaStream_t);  \
    template cudaError_t launch_layer_norm_backward<T>(                                           \
        const void *, const void *, const void *, const float *, const float *, void *, void *,   \
        void *, float *, const NormArgs &, cudaStream_t);
GS_NORM_INST(float)
GS_NORM_INST(__half)
GS_NORM_INST(__nv_bfloat16)
#undef GS_NORM_INST

}  // namespace gs
