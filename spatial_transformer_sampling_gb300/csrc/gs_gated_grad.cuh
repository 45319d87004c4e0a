// gs_gated_grad.cuh -- the gradients of both projections' outputs, dG = dH U act'(G)
// and dU = dH act(G), and the column sums that are the biases' gradients.
#pragma once

#include "gs_gated.cuh"

namespace gs {

// Bound by memory: three reads and two writes of rows x F.  A warp covers 32 V
// columns of a row; the block's eight warps walk rows, and its sums over them stay
// in registers until the end.
constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32;

// fp32 as three bf16 numbers, each the nearest to what the ones before leave: their
// sum is x to 2^-24 of it or better.  What is not finite stays in the first.
__device__ __forceinline__ void split3(float x, __nv_bfloat16 (&v)[3]) {
    v[0] = __float2bfloat16_rn(x);
    if (__hisinf(v[0])) v[0] = __float2bfloat16_rz(x);   // the largest numbers round to infinity
    const float r = isfinite(x) ? x - __bfloat162float(v[0]) : 0.0f;
    v[1] = __float2bfloat16_rn(r);
    v[2] = __float2bfloat16_rn(r - __bfloat162float(v[1]));
}

// Stores a run where the products read it: rounded to the type, or, of fp32, in three
// planes `plane` elements apart.
template <typename T> using Factor = std::conditional_t<sizeof(T) == 4, __nv_bfloat16, T>;
template <typename T, int V>
__device__ __forceinline__ void store_factor(Factor<T> *to, int64_t plane, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
        struct alignas(V * 2) Part { __nv_bfloat16 e[V]; } part[3];
#pragma unroll
        for (int e = 0; e < V; ++e) {
            __nv_bfloat16 x[3];
            split3(v[e], x);
#pragma unroll
            for (int i = 0; i < 3; ++i) part[i].e[e] = x[i];
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<Part *>(to + i * plane) = part[i];
    } else {
        Run<T, V>::store(to, v);
    }
}

inline int gated_grad_col_blocks(int F, int V) { return (F + 32 * V - 1) / (32 * V); }
// Row blocks: about four blocks of 256 threads per SM.
inline int gated_grad_row_blocks(int64_t rows, int F, int V) {
    const int cols = gated_grad_col_blocks(F, V);
    const int64_t most = (4 * kGatedSms + cols - 1) / cols, need = (rows + kGradWarps - 1) / kGradWarps;
    return (int)(need < most ? need : most);
}

// Into dG and dU (rows, pitch), planes of fp32 rows * pitch apart, and, with SUMS,
// partials[row block][2][F].
template <typename T, int V, bool SUMS, int ACT>
__device__ __forceinline__ void gated_grad_rows(const GatedArgs &a, const T *dH, const T *G,
                                                const T *U, Factor<T> *dG, Factor<T> *dU,
                                                int64_t pitch, float *partials) {
    using IOV = Run<T, V>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int f = (blockIdx.x * 32 + lane) * V;
    float sg[V] = {}, su[V] = {};
    if (f < a.F) {
#pragma unroll 2
        for (int64_t r = (int64_t)blockIdx.y * kGradWarps + warp; r < a.rows;
             r += (int64_t)gridDim.y * kGradWarps) {
            const int64_t at = r * a.F + f;
            float h[V], g[V], u[V];
            IOV::widen(IOV::load(dH + at), h);
            IOV::widen(IOV::load(G + at), g);
            IOV::widen(IOV::load(U + at), u);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float y, slope;
                act_and_slope<ACT>(g[e], y, slope);
                g[e] = h[e] * u[e] * slope;
                u[e] = h[e] * y;
                if (SUMS) {
                    sg[e] += g[e];
                    su[e] += u[e];
                }
            }
            store_factor<T, V>(dG + r * pitch + f, a.rows * pitch, g);
            store_factor<T, V>(dU + r * pitch + f, a.rows * pitch, u);
        }
    }
    if (!SUMS) return;
    __shared__ float s[2][kGradWarps][32 * V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        s[0][warp][lane * V + e] = sg[e];
        s[1][warp][lane * V + e] = su[e];
    }
    __syncthreads();
    float *out = partials + (int64_t)blockIdx.y * 2 * a.F;
    for (int c = threadIdx.x; c < 32 * V; c += kGradThreads) {
        const int d = blockIdx.x * 32 * V + c;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) {
            t0 += s[0][w][c];
            t1 += s[1][w][c];
        }
        if (d < a.F) {
            out[d] = t0;
            out[a.F + d] = t1;
        }
    }
}

template <typename T, int V, bool SUMS>
__global__ void __launch_bounds__(kGradThreads)
    gated_grad_kernel(GatedArgs a, const T *dH, const T *G, const T *U, Factor<T> *dG, Factor<T> *dU,
                      int64_t pitch, float *partials) {
    with_act(a.act, [&](auto act) {
        gated_grad_rows<T, V, SUMS, decltype(act)::value>(a, dH, G, U, dG, dU, pitch, partials);
    });
}

template <typename T, int V>
cudaError_t launch_gated_grad(const GatedArgs &a, const GatedPtrs &p, Factor<T> *dG, Factor<T> *dU,
                              int64_t pitch, float *partials, cudaStream_t s) {
    const dim3 grid(gated_grad_col_blocks(a.F, V), gated_grad_row_blocks(a.rows, a.F, V));
    const auto kernel = p.dbg ? gated_grad_kernel<T, V, true> : gated_grad_kernel<T, V, false>;
    kernel<<<grid, kGradThreads, 0, s>>>(a, (const T *)p.dH, (const T *)p.G, (const T *)p.U, dG, dU,
                                         pitch, partials);
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
