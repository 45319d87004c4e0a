// gs_gated_launch.cuh -- workspace layout and launches of the gated projections.
#pragma once

#include "gs_gated_grad.cuh"
#include "gs_gated_simt.cuh"

namespace gs {

// Workspace of the backward pass: dG and dU, then the biases' partial sums.
template <typename T> struct GatedLayout {
    int64_t pitch;
    size_t dG, dU, partials, bytes;
    explicit GatedLayout(const GatedArgs &a) {
        const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
        pitch = (a.F + 7) / 8 * 8;
        dG = 0;
        dU = up((size_t)a.rows * pitch * sizeof(T));
        partials = 2 * dU;
        // whatever the alignment will be
        const int b1 = gated_grad_row_blocks(a.rows, a.F, 1);
        const int bv = gated_grad_row_blocks(a.rows, a.F, kVec<T>);
        bytes = partials + up((size_t)(b1 > bv ? b1 : bv) * 2 * a.F * sizeof(float));
    }
};

template <typename T> size_t gated_ws_bytes(const GatedArgs &a, bool backward) {
    if (!backward || a.rows == 0 || a.F == 0) return 0;
    return GatedLayout<T>(a).bytes;
}

template <typename T>
cudaError_t launch_gated(const GatedArgs &a, const GatedPtrs &p, void *, cudaStream_t s) {
    gated_simt_kernel<T><<<(unsigned)simt_blocks(a.rows, a.F), kSimtThreads, 0, s>>>(a, p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gated_backward(const GatedArgs &a, const GatedPtrs &p, void *ws,
                                  cudaStream_t s) {
    const GatedLayout<T> at(a);
    char *base = (char *)ws;
    T *dG = (T *)(base + at.dG), *dU = (T *)(base + at.dU);
    float *partials = (float *)(base + at.partials);
    const bool wide = a.F % kVec<T> == 0 && aligned16(p.dH) && aligned16(p.G) && aligned16(p.U);
    cudaError_t e = wide ? launch_gated_grad<T, kVec<T>>(a, p, dG, dU, at.pitch, partials, s)
                         : launch_gated_grad<T, 1>(a, p, dG, dU, at.pitch, partials, s);
    if (e != cudaSuccess) return e;
    if (p.dbg) {
        const int blocks = gated_grad_row_blocks(a.rows, a.F, wide ? kVec<T> : 1);
        e = launch_gated_bias_sums<T>(a, p, partials, blocks, true, s);
        if (e != cudaSuccess) return e;
    }
    const auto product = [&](SimtProduct q, void *out) {
        return launch_next(true, gated_simt_product_kernel<T>, dim3((unsigned)simt_blocks(q.M, q.N)),
                           kSimtThreads, 0, s, q, (T *)out);
    };
    e = product({{dG, dU}, {p.Wg, p.Wu}, at.pitch, 1, 1, a.D, a.rows, a.D, a.F, 2}, p.dX);
    if (e != cudaSuccess) return e;
    e = product({{dG, dG}, {p.X, p.X}, 1, at.pitch, 1, a.D, a.F, a.D, a.rows, 1}, p.dWg);
    if (e != cudaSuccess) return e;
    return product({{dU, dU}, {p.X, p.X}, 1, at.pitch, 1, a.D, a.F, a.D, a.rows, 1}, p.dWu);
}

#define GS_GATED_INST(T)                                                                         \
    template size_t gated_ws_bytes<T>(const GatedArgs &, bool);                                   \
    template cudaError_t launch_gated<T>(const GatedArgs &, const GatedPtrs &, void *,            \
                                         cudaStream_t);                                           \
    template cudaError_t launch_gated_backward<T>(const GatedArgs &, const GatedPtrs &, void *,   \
                                                  cudaStream_t);

}  // namespace gs
