// gs_gated_grad.cuh -- the gradients of both projections' outputs, dG = dH U act'(G)
// and dU = dH act(G), and the column sums that are the biases' gradients.
#pragma once

#include <initializer_list>

#include "gs_gated.cuh"

namespace gs {

// Bound by memory: three reads and two writes of rows x F.  A team of 8, 16 or 32 lanes
// covers as many runs of a row; the block's teams walk rows, and a lane's sums over them
// stay in registers until the end.
constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32;

// How the rows are gone over: lanes of a team, blocks along F and along the rows (about
// four blocks of 256 threads per SM).
struct GradPlan {
    int team, cols, rows;
};
inline GradPlan grad_plan(int64_t rows, int F, int V) {
    const int runs = (F + V - 1) / V, team = runs <= 8 ? 8 : runs <= 16 ? 16 : 32;
    const int cols = (runs + team - 1) / team, each = kGradThreads / team;
    const int64_t most = (4 * kGatedSms + cols - 1) / cols, need = (rows + each - 1) / each;
    return {team, cols, (int)(need < most ? need : most)};
}

// fp32 as three bf16 numbers, each the nearest to what the ones before leave: their
// sum is x to 2^-24 of it or better.  What is not finite stays in the first.  Two at a
// time, packed.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void split3(float lo, float hi, uint32_t (&v)[3]) {
    v[0] = bf16_pair(lo, hi);
    float a = __uint_as_float(v[0] << 16), b = __uint_as_float(v[0] & 0xffff0000u);
    if (!(fabsf(a) < INFINITY) || !(fabsf(b) < INFINITY)) {
        // NaN and infinities leave nothing; the largest numbers do not round to infinity
        if (isinf(a) && !isinf(lo)) a = copysignf(3.3895314e38f, lo);
        if (isinf(b) && !isinf(hi)) b = copysignf(3.3895314e38f, hi);
        v[0] = bf16_pair(a, b);
        if (!isfinite(lo)) lo = a = 0.0f;
        if (!isfinite(hi)) hi = b = 0.0f;
    }
    lo -= a;
    hi -= b;
    v[1] = bf16_pair(lo, hi);
    v[2] = bf16_pair(lo - __uint_as_float(v[1] << 16), hi - __uint_as_float(v[1] & 0xffff0000u));
}

// kVec<T> elements from element e of a tensor of `total`, whatever e: the two 16-byte
// runs that hold them, shifted together.  The tensor starts on a 16-byte boundary; what
// lies behind its end reads as 0.
template <typename T>
__device__ __forceinline__ uint4 load_shifted(const T *base, int64_t e, int64_t total) {
    constexpr int V = kVec<T>;
    const int64_t run = e / V * V;
    const int by = (int)(e - run);
    if (run + 2 * V <= total || (by == 0 && run + V <= total)) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(base + run));
        if (by == 0) return a;
        const uint4 b = __ldg(reinterpret_cast<const uint4 *>(base + run + V));
        uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const int words = by * (int)sizeof(T) / 4;
        if (words & 2) {
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
        }
        if (words & 1) {
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
        }
        if (sizeof(T) == 2 && (by & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    uint4 v;
    T *x = reinterpret_cast<T *>(&v);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = e + i < total ? base[e + i] : IO<T>::st(0.0f);
    return v;
}

// How rows are read: one element at a time, in 16-byte runs, or in runs that start
// anywhere (rows that are no multiple of 16 bytes in a tensor that starts on one).
enum { kRowsSingle = 0, kRowsRuns = 1, kRowsShifted = 2 };
template <typename T, int READ> constexpr int kRowsV = READ == kRowsSingle ? 1 : kVec<T>;
template <typename T, int READ>
__device__ __forceinline__ typename Run<T, kRowsV<T, READ>>::Raw row_load(const T *base, int64_t e,
                                                                          int64_t total) {
    if constexpr (READ == kRowsShifted)
        return load_shifted(base, e, total);
    else
        return Run<T, kRowsV<T, READ>>::load(base + e);
}
template <typename T> int rows_read(int width, std::initializer_list<const void *> tensors) {
    for (const void *t : tensors)
        if (!aligned16(t)) return kRowsSingle;
    return width % kVec<T> == 0 ? kRowsRuns : kRowsShifted;
}

// Stores a run where the products read it: rounded to the type, or, of fp32, in three
// planes `plane` elements apart.  In 16-bit types that rounding shows in the products (2.3e-3
// of them in bf16 and 2.9e-4 in fp16, 1.7e-3 and 2.1e-4 by the store alone): a second plane
// would take it away for twice the products, which are 289 of the 414 us of 16384 x 1024 x 4096.
template <typename T> using Factor = std::conditional_t<sizeof(T) == 4, __nv_bfloat16, T>;
template <typename T, int V>
__device__ __forceinline__ void store_factor(Factor<T> *to, int64_t plane, const float (&v)[V]) {
    static_assert(sizeof(T) == 2 || V == 1 || V == 4, "a run of fp32");
    if constexpr (sizeof(T) == 4) {
        uint32_t x[3], y[3] = {};
        split3(v[0], V > 1 ? v[V > 1 ? 1 : 0] : 0.0f, x);
        if constexpr (V == 4) split3(v[2], v[3], y);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(to + i * plane) = make_uint2(x[i], y[i]);
            else
                to[i * plane] = __ushort_as_bfloat16((unsigned short)x[i]);
        }
    } else {
        Run<T, V>::store(to, v);
    }
}

// In fp16 dG and dU are scaled by a power of two, so that as factors of the products they
// do not leave the type's range: 2^14 over the power of two below `bound`, the largest
// finite |dG| or |dU| of the call.  What is 2^-28 of that or more keeps the type's
// precision; smaller elements are off by up to 2^-39 of it.
// Finding it takes one more pass over the inputs, which forms dG and dU as the next one
// does: a bound from |dH|, |U| and |G| would let rows far out, whose slopes are 0, take
// the others' digits (gelu, 16384 x 1024 x 4096, the whole call 488 us, and 480 by a bound).
// The second pass finds up to 100 MB of the inputs in L2.
__device__ __forceinline__ float gated_scale(uint32_t bound, bool inverse) {
    const int e = (int)(bound >> 23) - 127;            // of a number that is not negative
    if (bound == 0) return 1.0f;                       // nothing
    const int s = max(-100, min(100, inverse ? e - 14 : 14 - e));
    return __int_as_float((s + 127) << 23);
}
template <typename T, int READ>
__global__ void __launch_bounds__(kGradThreads)
    gated_bound_kernel(GatedArgs a, const T *dH, const T *G, const T *U, uint32_t *bound) {
    constexpr int V = kRowsV<T, READ == kRowsSingle ? kRowsSingle : kRowsRuns>;
    using IOV = Run<T, V>;
    const int64_t total = a.rows * a.F, runs = total / V;
    float most = 0.0f;
    with_act(a.act, [&](auto act) {
        // what is not finite is left out, so that it does not reach the scale of other rows
        const auto take = [&](float h, float g, float u) {
            float y, slope;
            act_and_slope<T, decltype(act)::value>(g, y, slope);
            const float dg = fabsf(h * u * slope), du = fabsf(h * y);
            most = fmaxf(most, fmaxf(dg < INFINITY ? dg : 0.0f, du < INFINITY ? du : 0.0f));
        };
        // the rows are one array here
#pragma unroll 2
        for (int64_t i = (int64_t)blockIdx.x * kGradThreads + threadIdx.x; i < runs;
             i += (int64_t)gridDim.x * kGradThreads) {
            float h[V], g[V], u[V];
            IOV::widen(IOV::load(dH + i * V), h);
            IOV::widen(IOV::load(G + i * V), g);
            IOV::widen(IOV::load(U + i * V), u);
#pragma unroll
            for (int e = 0; e < V; ++e) take(h[e], g[e], u[e]);
        }
        if (blockIdx.x == 0 && runs * V + threadIdx.x < total) {
            const int64_t e = runs * V + threadIdx.x;
            take(IO<T>::ld(dH + e), IO<T>::ld(G + e), IO<T>::ld(U + e));
        }
    });
    // a maximum does not depend on the order, and numbers that are not negative compare
    // as their bits do
    __shared__ float warps[kGradWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = most;
    __syncthreads();
    if (threadIdx.x > 0) return;
#pragma unroll
    for (int w = 1; w < kGradWarps; ++w) most = fmaxf(most, warps[w]);
    atomicMax(bound, __float_as_uint(most));
}
template <typename T>
cudaError_t launch_gated_bound(const GatedArgs &a, const GatedPtrs &p, bool runs, uint32_t *bound,
                               cudaStream_t s) {
    const cudaError_t e = cudaMemsetAsync(bound, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return e;
    const int V = runs ? kVec<T> : 1;
    const int64_t need = (a.rows * a.F / V + kGradThreads - 1) / kGradThreads;
    const unsigned blocks = (unsigned)(need < 8 * kGatedSms ? (need > 0 ? need : 1) : 8 * kGatedSms);
    const auto kernel = runs ? gated_bound_kernel<T, kRowsRuns> : gated_bound_kernel<T, kRowsSingle>;
    kernel<<<blocks, kGradThreads, 0, s>>>(a, (const T *)p.dH, (const T *)p.G, (const T *)p.U, bound);
    return cudaGetLastError();
}

// Into dG and dU (rows, pitch), planes of fp32 rows * pitch apart, and, with SUMS,
// partials[row block][2][F].
template <typename T, int READ, bool SUMS, int ACT>
__device__ __forceinline__ void gated_grad_rows(const GatedArgs &a, const T *dH, const T *G,
                                                const T *U, Factor<T> *dG, Factor<T> *dU,
                                                int64_t pitch, float *partials, int team, float scale,
                                                float (*s)[kGradWarps][32 * kRowsV<T, READ>]) {
    constexpr int V = kRowsV<T, READ>;
    using IOV = Run<T, V>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, teams = kGradThreads / team;
    const int64_t total = a.rows * a.F;
    const int f = (blockIdx.x * team + threadIdx.x % team) * V;
    float sg[V] = {}, su[V] = {};
    if (f < a.F) {
#pragma unroll 2
        for (int64_t r = (int64_t)blockIdx.y * teams + threadIdx.x / team; r < a.rows;
             r += (int64_t)gridDim.y * teams) {
            const int64_t at = r * a.F + f;
            float h[V], g[V], u[V];
            IOV::widen(row_load<T, READ>(dH, at, total), h);
            IOV::widen(row_load<T, READ>(G, at, total), g);
            IOV::widen(row_load<T, READ>(U, at, total), u);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float y, slope;
                act_and_slope<T, ACT>(g[e], y, slope);
                g[e] = h[e] * u[e] * slope;
                u[e] = h[e] * y;
                if (SUMS) {
                    sg[e] += g[e];
                    su[e] += u[e];
                }
            }
            if (__is_same(T, __half)) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    g[e] *= scale;
                    u[e] *= scale;
                }
            }
            store_factor<T, V>(dG + r * pitch + f, a.rows * pitch, g);
            store_factor<T, V>(dU + r * pitch + f, a.rows * pitch, u);
        }
    }
    if (!SUMS) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s[0][warp][lane * V + e] = sg[e];
        s[1][warp][lane * V + e] = su[e];
    }
    __syncthreads();
    float *out = partials + (int64_t)blockIdx.y * 2 * a.F;
    // the teams in order
    const float *all_g = &s[0][0][0], *all_u = &s[1][0][0];
    for (int c = threadIdx.x; c < team * V; c += kGradThreads) {
        const int d = blockIdx.x * team * V + c;
        float t0 = 0.0f, t1 = 0.0f;
        for (int w = 0; w < teams; ++w) {
            t0 += all_g[w * team * V + c];
            t1 += all_u[w * team * V + c];
        }
        if (d < a.F) {
            out[d] = t0;
            out[a.F + d] = t1;
        }
    }
}

template <typename T, int READ, bool SUMS>
__global__ void __launch_bounds__(kGradThreads, 3)
    gated_grad_kernel(GatedArgs a, const T *dH, const T *G, const T *U, Factor<T> *dG, Factor<T> *dU,
                      int64_t pitch, float *partials, int team, const uint32_t *bound) {
    const float scale = __is_same(T, __half) ? gated_scale(__ldg(bound), false) : 1.0f;
    __shared__ float sums[SUMS ? 2 : 1][SUMS ? kGradWarps : 1][32 * kRowsV<T, READ>];
    with_act(a.act, [&](auto act) {
        gated_grad_rows<T, READ, SUMS, decltype(act)::value>(
            a, dH, G, U, dG, dU, pitch, partials, team, scale,
            reinterpret_cast<float(*)[kGradWarps][32 * kRowsV<T, READ>]>(sums));
    });
}

template <typename T, int READ>
cudaError_t launch_gated_grad(const GatedArgs &a, const GatedPtrs &p, Factor<T> *dG, Factor<T> *dU,
                              int64_t pitch, float *partials, const uint32_t *bound,
                              cudaStream_t s) {
    constexpr int V = kRowsV<T, READ>;
    const GradPlan plan = grad_plan(a.rows, a.F, V);
    const auto kernel = p.dbg ? gated_grad_kernel<T, READ, true> : gated_grad_kernel<T, READ, false>;
    kernel<<<dim3(plan.cols, plan.rows), kGradThreads, 0, s>>>(
        a, (const T *)p.dH, (const T *)p.G, (const T *)p.U, dG, dU, pitch, partials, plan.team, bound);
    return cudaGetLastError();
}

// The biases' gradients from the partial sums; without rows, zeros.
template <typename T>
cudaError_t launch_gated_bias_sums(const GatedArgs &a, const GatedPtrs &p, const float *partials,
                                   int blocks, bool follows, cudaStream_t s) {
    SumArgs sums = {};
    sums.from = partials;
    sums.to[0] = p.dbg;
    sums.to[1] = p.dbu;
    sums.vectors = 2;
    sums.count = blocks;
    sums.pitch = 2 * (int64_t)a.F;
    sums.D = a.F;
    return launch_sums<T>(sums, follows, s);
}

}  // namespace gs
