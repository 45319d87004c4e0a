// gs_dropout.cu -- dropout from a counter-based generator, with an optional
// residual sum: Y = residual + (kept ? X / (1 - ratio) : 0).
//
// The mask is a function of (seed, offset, element index) and is never stored:
// the backward pass calls the same kernel on the gradient.  A thread moves
// 16-byte runs, kRuns of them a block apart, all loads first.  For 16-bit types
// the generator weighs as much as the memory traffic (18 wide products and 20
// exclusive-ors per four elements): 67 M bf16 with a residual take 63.2 us (6.4
// TB/s), 33.5 M fp16 without one 26.9 us (5.0 TB/s).  Two runs per thread in 32
// registers took a fifth more.
#include "gs_internal.h"
#include "gs_philox.cuh"
#include "gs_ptx.cuh"
#include "gs_vec.cuh"

namespace gs {
namespace {

constexpr int kDropThreads = 256;
constexpr int kRuns = 4;

// The kept and scaled value of E consecutive elements from element 4 * quad on
// (`high`: bits 32 and up of quad), plus r.
template <int E, bool RES>
__device__ __forceinline__ void drop(float (&x)[E], const float (&r)[E], uint32_t quad, uint32_t high,
                                     const DropoutArgs &a, const PhiloxKeys &keys) {
    const float2 scale = make_float2(a.scale, a.scale);
#pragma unroll
    for (int e = 0; e < E; e += 4) {
        uint32_t w[4];
        philox4x32_10(quad + e / 4, high, a.offset, keys, w);
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
            float2 y = mul_f32x2(make_float2(x[e + q], x[e + q + 1]), scale);
            y.x = w[q] >= a.threshold ? y.x : 0.0f;
            y.y = w[q + 1] >= a.threshold ? y.y : 0.0f;
            if (RES) y = add_f32x2(make_float2(r[e + q], r[e + q + 1]), y);
            x[e + q] = y.x;
            x[e + q + 1] = y.y;
        }
    }
}

// Runs of 16 bytes (VEC), or where a base is not aligned and at the end of the
// tensor four elements (one generator call) moved one by one.  X, residual and
// Y may be the same memory: a thread reads an element before it writes it, and
// no other does.
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(kDropThreads)
    dropout_kernel(const T *X, const T *residual, T *Y, DropoutArgs a,
                   const __grid_constant__ PhiloxKeys keys) {
    constexpr int E = VEC ? kVec<T> : 4;
    const int64_t run0 = (int64_t)blockIdx.x * (kDropThreads * kRuns) + threadIdx.x;
    // a block's generator calls share their upper 32 bits: it makes a power of
    // two of them, aligned to that
    const uint64_t first = (uint64_t)blockIdx.x * (kDropThreads * kRuns * (E / 4));
    const uint32_t high = (uint32_t)(first >> 32);
    if constexpr (VEC) {
        if ((run0 + (kRuns - 1) * kDropThreads + 1) * E <= a.n) {
            using IOV = Run<T, E>;
            typename IOV::Raw rx[kRuns], rr[kRuns];
#pragma unroll
            for (int k = 0; k < kRuns; ++k) {
                const int64_t i = (run0 + k * kDropThreads) * E;
                rx[k] = IOV::load(X + i);
                if (RES) rr[k] = IOV::load(residual + i);
            }
#pragma unroll
            for (int k = 0; k < kRuns; ++k) {
                const int64_t i = (run0 + k * kDropThreads) * E;
                float x[E], r[E];
                IOV::widen(rx[k], x);
                if (RES) IOV::widen(rr[k], r);
                drop<E, RES>(x, r, (uint32_t)(i / 4), high, a, keys);
                IOV::store(Y + i, x);
            }
            return;
        }
    }
#pragma unroll 1
    for (int k = 0; k < kRuns; ++k)
#pragma unroll 1
        for (int part = 0; part < E; part += 4) {
            const int64_t i = (run0 + k * kDropThreads) * E + part;
            float x[4], r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = i + e < a.n ? IO<T>::to_f(X[i + e]) : 0.0f;
                r[e] = RES && i + e < a.n ? IO<T>::to_f(residual[i + e]) : 0.0f;
            }
            if (i >= a.n) return;
            drop<4, RES>(x, r, (uint32_t)(i / 4), high, a, keys);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < a.n) Y[i + e] = IO<T>::st(x[e]);
        }
}

}  // namespace

template <typename T>
cudaError_t launch_dropout(const void *X, const void *residual, void *Y, const DropoutArgs &a,
                           cudaStream_t s) {
    const bool vec = aligned16(X) && aligned16(residual) && aligned16(Y);
    const int64_t per_block = (int64_t)kDropThreads * kRuns * (vec ? kVec<T> : 4);
    auto kernel = residual ? (vec ? dropout_kernel<T, true, true> : dropout_kernel<T, false, true>)
                           : (vec ? dropout_kernel<T, true, false> : dropout_kernel<T, false, false>);
    kernel<<<(unsigned)((a.n + per_block - 1) / per_block), kDropThreads, 0, s>>>(
        (const T *)X, (const T *)residual, (T *)Y, a, philox_keys(a.seed));
    return cudaGetLastError();
}

template cudaError_t launch_dropout<float>(const void *, const void *, void *, const DropoutArgs &,
                                           cudaStream_t);
template cudaError_t launch_dropout<__half>(const void *, const void *, void *, const DropoutArgs &,
                                            cudaStream_t);
template cudaError_t launch_dropout<__nv_bfloat16>(const void *, const void *, void *,
                                                   const DropoutArgs &, cudaStream_t);

}  // namespace gs
