// gs_gated_grad.cuh -- the gradients of both projections' outputs, dG = dH U act'(G)
// and dU = dH act(G), and the column sums that are the biases' gradients.
#pragma once

#include "gs_gated.cuh"

namespace gs {

// Bound by memory: three reads and two writes of rows x F.  A warp covers 32 V
// columns of a row; the block's eight warps walk rows, and its sums over them stay
// in registers until the end.
constexpr int kGradThreads = 256, kGradWarps = kGradThreads / 32;

inline int gated_grad_col_blocks(int F, int V) { return (F + 32 * V - 1) / (32 * V); }
// Row blocks: about four blocks of 256 threads per SM.
inline int gated_grad_row_blocks(int64_t rows, int F, int V) {
    const int cols = gated_grad_col_blocks(F, V);
    const int64_t most = (4 * kGatedSms + cols - 1) / cols, need = (rows + kGradWarps - 1) / kGradWarps;
    return (int)(need < most ? need : most);
}

// Into dG and dU (rows, pitch) and, with SUMS, partials[row block][2][F].
template <typename T, int V, bool SUMS, int ACT>
__device__ __forceinline__ void gated_grad_rows(const GatedArgs &a, const T *dH, const T *G,
                                                const T *U, T *dG, T *dU, int64_t pitch,
                                                float *partials) {
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
            IOV::store(dG + r * pitch + f, g);
            IOV::store(dU + r * pitch + f, u);
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
    gated_grad_kernel(GatedArgs a, const T *dH, const T *G, const T *U, T *dG, T *dU, int64_t pitch,
                      float *partials) {
    with_act(a.act, [&](auto act) {
        gated_grad_rows<T, V, SUMS, decltype(act)::value>(a, dH, G, U, dG, dU, pitch, partials);
    });
}

template <typename T, int V>
cudaError_t launch_gated_grad(const GatedArgs &a, const GatedPtrs &p, T *dG, T *dU, int64_t pitch,
                              float *partials, cudaStream_t s) {
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
