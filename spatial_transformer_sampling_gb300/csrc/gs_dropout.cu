// gs_dropout.cu -- dropout from a counter-based generator, with an optional
// residual sum: Y = residual + (kept ? X / (1 - ratio) : 0).
//
// The mask is a function of (seed, offset, element index) and is never stored:
// the backward pass calls the same kernel on the gradient.
#include "gs_common.cuh"
#include "gs_internal.h"
#include "gs_philox.cuh"

namespace gs {

template <typename T>
__global__ void dropout_kernel(const T *X, const T *residual, T *Y, DropoutArgs a) {
    const int64_t quad = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t i0 = quad * 4;
    if (i0 >= a.n) return;
    uint32_t w[4];
    philox4x32_10((uint64_t)quad, a.offset, a.seed, w);
    for (int k = 0; k < 4 && i0 + k < a.n; ++k) {
        const float x = IO<T>::to_f(X[i0 + k]);
        float y = w[k] >= a.threshold ? x * a.scale : 0.0f;
        if (residual) y += IO<T>::to_f(residual[i0 + k]);
        Y[i0 + k] = IO<T>::st(y);
    }
}

template <typename T>
cudaError_t launch_dropout(const void *X, const void *residual, void *Y, const DropoutArgs &a,
                           cudaStream_t s) {
    const int64_t blocks = ((a.n + 3) / 4 + 255) / 256;
    dropout_kernel<T><<<(unsigned)blocks, 256, 0, s>>>((const T *)X, (const T *)residual, (T *)Y, a);
    return cudaGetLastError();
}

template cudaError_t launch_dropout<float>(const void *, const void *, void *, const DropoutArgs &,
                                           cudaStream_t);
template cudaError_t launch_dropout<__half>(const void *, const void *, void *, const DropoutArgs &,
                                            cudaStream_t);
template cudaError_t launch_dropout<__nv_bfloat16>(const void *, const void *, void *,
                                                   const DropoutArgs &, cudaStream_t);

}  // namespace gs
