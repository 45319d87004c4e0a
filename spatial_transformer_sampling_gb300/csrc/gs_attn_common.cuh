// gs_attn_common.cuh -- what the attention kernels share: token geometry, the
// expanded bias and the base-2 exponential.
#pragma once

#include "gs_common.cuh"
#include "gs_internal.h"

namespace gs {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the hardware instruction, results below 2^-126 as 0: an fp32 gradient is
// off by 5.1e-7 of its size with it, by 4.8e-7 with exp in fp32.  x = -inf gives 0.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Relative index of a token on its side (see AttnArgs).
__device__ __forceinline__ int rel_q(const AttnArgs &a, int i) {
    const int y = i / a.Wq;
    return (y + a.Hk - 1) * a.P + (i - y * a.Wq) + a.Wk - 1;
}
__device__ __forceinline__ int rel_k(const AttnArgs &a, int j) {
    const int y = j / a.Wk;
    return y * a.P + (j - y * a.Wk);
}

// Keys of batch item n that may be attended to.
__device__ __forceinline__ int keys_of(const AttnArgs &a, int n) {
    return a.k_len ? min(max(__ldg(a.k_len + n), 0), a.Lk) : a.Lk;
}

// One bias entry in base-2 units: table[b][h] * log2(e), -inf where the bucket
// lies outside the table (the pair is masked).  A finite entry stays finite:
// the lowest value of a type times log2(e) would leave fp32's range, and a row
// of such entries is a uniform softmax, not an empty one.
__device__ __forceinline__ float bias2(float b) {
    const float f = b * kLog2e;
    return isinf(f) && !isinf(b) ? copysignf(3.4028234e38f, b) : f;
}

// A row's LSE in base 2, from which the backward pass subtracts its scores; a row
// with no key: weights of 0.  The same steps as a table entry's: in a row of one
// common entry, however large, the two cancel.
__device__ __forceinline__ float lse2_of(float lse) { return lse == -INFINITY ? INFINITY : bias2(lse); }

// A row's LSE from t = m + log2 l where the spacing of t is no longer small beside
// 1: the lowest number with lse2_of(LSE) >= t, one step from t / log2 e at most.  One
// lower, and the weights of the backward pass would be 2^128 and more for scores of
// -1e9.  Out of the kernels' way: in place it took 2 us more over 1024 windows of
// 8 x 8 (47 us).
static __device__ __noinline__ float lse_of_far(float t) {
    const float v = t * kLn2, lower = nextafterf(v, -INFINITY);
    return lse2_of(lower) >= t ? lower : lse2_of(v) < t ? nextafterf(v, INFINITY) : v;
}

// A row's LSE from the reference `m` of its scores and the sum `l` of 2^(s - m),
// 0 where there is no key.
__device__ __forceinline__ float lse_of(float m, float l) {
    const float t = l != 0.0f ? m + log2f(l) : -INFINITY;
    return fabsf(t) >= 1048576.0f && !isinf(t) ? lse_of_far(t) : t * kLn2;
}

template <typename T>
__device__ __forceinline__ float bias2_of(const T *table, int bucket, int nb, int H, int h) {
    if ((unsigned)bucket >= (unsigned)nb) return -INFINITY;
    return bias2(IO<T>::ld(table + (int64_t)bucket * H + h));
}

}  // namespace gs
