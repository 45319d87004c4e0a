// gs_gated.cuh -- the gated projections of a feed-forward block:
//   G = X Wg^T + bg, U = X Wu^T + bu, H = act(G) * U,
// and their gradient from dH, G and U:
//   dG = dH U act'(G), dU = dH act(G), dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X.
#pragma once

#include "../../include/gs.h"
#include "gs_attn_common.cuh"
#include "gs_sums.cuh"

namespace gs {

// 1 / (1 + e^-x): two hardware approximations of 2 ulps each.
__device__ __forceinline__ float sigmoid_of(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.0f + exp2_approx(-kLog2e * x)));
    return y;
}

// The tanh form's argument, doubled: 0.5 (1 + tanh a) = sigmoid(2 a).
constexpr float kGeluTanh2 = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluCubic = 0.044715f;

// The normal distribution's Phi(g), and *density = e^(-g^2 / 2).  With x = |g| / sqrt 2 and
// t = 1 / (1 + p x), Phi(-|g|) = t q(t) e^(-x^2), where q is the polynomial in t that is
// nearest to erfc(x) e^(x^2) / (2 t) on 0 <= x <= 9.6 in the largest relative error (found by
// reweighted least squares): 1.0e-6 of it with seven terms, for 16-bit types, and 6.7e-9 with
// ten, for fp32.  Relative to Phi, so that the negative tail keeps its digits where
// (1 + erf) / 2 cancels; behind 9.6 the exponential is 0.  It serves the slope as well
// (262144 x 64 x 256, kept, fp32 309 us, with erfcf 395; bf16 98, 95 with five terms that are
// off by 1.5e-7 of 1 and not of Phi).
template <typename T> __device__ __forceinline__ float normal_phi(float g, float *density) {
    constexpr bool kWide = sizeof(T) == 4;
    constexpr float p = (kWide ? 0.35f : 0.38f) * 0.70710678118654752f;
    *density = exp2_approx(-0.5f * kLog2e * g * g);
    float t, q;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(p, fabsf(g), 1.0f)));
    if (kWide) {
        q = fmaf(0.018888099f, t, -0.077709257f);
        q = fmaf(q, t, 0.086447849f);
        q = fmaf(q, t, -0.007902219f);
        q = fmaf(q, t, 0.038330668f);
        q = fmaf(q, t, 0.075943622f);
        q = fmaf(q, t, 0.074525383f);
        q = fmaf(q, t, 0.094194337f);
        q = fmaf(q, t, 0.098537903f);
        q = fmaf(q, t, 0.098743619f);
    } else {
        q = fmaf(-0.062540521f, t, 0.167370233f);
        q = fmaf(q, t, -0.033950628f);
        q = fmaf(q, t, 0.123114330f);
        q = fmaf(q, t, 0.090643001f);
        q = fmaf(q, t, 0.108212830f);
        q = fmaf(q, t, 0.107150248f);
    }
    const float tail = q * t * *density;   // Phi(-|g|)
    return g < 0.0f ? tail : 1.0f - tail;
}

// T: the type of the result.
template <typename T, int ACT> __device__ __forceinline__ float act_of(float g) {
    if (ACT == GS_ACT_SILU) return g * sigmoid_of(g);
    if (ACT == GS_ACT_GELU) {
        float density;
        return g * normal_phi<T>(g, &density);
    }
    if (ACT == GS_ACT_GELU_TANH) return g * sigmoid_of(kGeluTanh2 * g * fmaf(kGeluCubic * g, g, 1.0f));
    if (ACT == GS_ACT_RELU) return g < 0.0f ? 0.0f : g;   // NaN stays
    if (ACT == GS_ACT_SIGMOID) return sigmoid_of(g);
    return g;
}

// act(g) for a whole kernel, chosen by numbers where one formula serves: the sigmoid
// family is sigmoid(g (c1 + c2 g^2)), times g or not; relu and identity are the larger
// of g and a bound.  Six copies of an unrolled epilogue did not stay in the instruction
// cache.
struct ActNumbers {
    int form;          // 0 sigmoid family, 1 gelu, 2 bounded
    bool times_g;
    float c1, c2, low;
};
inline ActNumbers act_numbers(int act) {
    if (act == GS_ACT_GELU) return {1, true, 0.0f, 0.0f, 0.0f};
    if (act == GS_ACT_RELU) return {2, true, 0.0f, 0.0f, 0.0f};
    if (act == GS_ACT_IDENTITY) return {2, true, 0.0f, 0.0f, -__builtin_inff()};
    const bool cubic = act == GS_ACT_GELU_TANH;
    return {0, act != GS_ACT_SIGMOID, cubic ? kGeluTanh2 : 1.0f, cubic ? kGeluTanh2 * kGeluCubic : 0.0f,
            0.0f};
}
// g[i] = act(g[i]) u[i].
template <typename T, int N>
__device__ __forceinline__ void act_product(const ActNumbers &a, float (&g)[N], const float (&u)[N]) {
    if (a.form == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // the square is bounded: it may not make 0 * infinity of c2 = 0
            const float r = sigmoid_of(g[i] * fmaf(a.c2, fminf(g[i] * g[i], 1e30f), a.c1));
            g[i] = (a.times_g ? g[i] * r : r) * u[i];
        }
    } else if (a.form == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = act_of<T, GS_ACT_GELU>(g[i]) * u[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) g[i] = (g[i] < a.low ? a.low : g[i]) * u[i];   // NaN stays
    }
}

// act(g) and its slope.
template <typename T, int ACT> __device__ __forceinline__ void act_and_slope(float g, float &a, float &da) {
    if (ACT == GS_ACT_SILU) {
        const float r = sigmoid_of(g);
        a = g * r;
        da = fmaf(a, 1.0f - r, r);
    } else if (ACT == GS_ACT_GELU) {
        float density;
        const float phi = normal_phi<T>(g, &density);
        a = g * phi;
        da = fmaf(g * 0.3989422804014327f, density, phi);
    } else if (ACT == GS_ACT_GELU_TANH) {
        // the square is bounded: it may not make 0 * infinity of 1 - r = 0
        const float g2 = fminf(g * g, 1e30f), r = sigmoid_of(kGeluTanh2 * g * fmaf(kGeluCubic, g2, 1.0f));
        a = g * r;
        da = fmaf(a * (1.0f - r), kGeluTanh2 * fmaf(3.0f * kGeluCubic, g2, 1.0f), r);
    } else if (ACT == GS_ACT_RELU) {
        a = g < 0.0f ? 0.0f : g;
        da = g > 0.0f ? 1.0f : 0.0f;
    } else if (ACT == GS_ACT_SIGMOID) {
        a = sigmoid_of(g);
        da = a * (1.0f - a);
    } else {
        a = g;
        da = 1.0f;
    }
}

// Calls f with the activation as a compile-time number.
template <typename F> __device__ __forceinline__ void with_act(int act, F &&f) {
    using std::integral_constant;
    switch (act) {
        case GS_ACT_SILU: f(integral_constant<int, GS_ACT_SILU>()); break;
        case GS_ACT_GELU: f(integral_constant<int, GS_ACT_GELU>()); break;
        case GS_ACT_GELU_TANH: f(integral_constant<int, GS_ACT_GELU_TANH>()); break;
        case GS_ACT_RELU: f(integral_constant<int, GS_ACT_RELU>()); break;
        case GS_ACT_SIGMOID: f(integral_constant<int, GS_ACT_SIGMOID>()); break;
        default: f(integral_constant<int, GS_ACT_IDENTITY>()); break;
    }
}

constexpr int kGatedSms = 152;

}  // namespace gs
