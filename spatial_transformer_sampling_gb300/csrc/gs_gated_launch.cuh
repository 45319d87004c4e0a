// gs_gated_launch.cuh -- workspace layout and launches of the gated projections.
#pragma once

#include "gs_gated_grad.cuh"
#include "gs_gated_simt.cuh"
#include "gs_gated_tc.cuh"

namespace gs {

// Rows of a matrix copied to a pitch of whole 16-byte runs; what lies behind a row's
// end is not written (and not read: the tensor maps end with the row).
template <typename T>
__global__ void __launch_bounds__(256) gated_pad_kernel(const T *from, T *to, int64_t n, int width,
                                                        int64_t pitch) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / width;
        to[r * pitch + (i - r * width)] = from[i];
    }
}

// Workspace: copies of X, Wg and Wu where rows are no multiple of 16 bytes; backward,
// dG and dU and the biases' partial sums.
template <typename T> struct GatedLayout {
    int64_t pitch_d, pitch_f;
    bool pad;
    size_t X, Wg, Wu, dG, dU, partials, bytes;
    GatedLayout(const GatedArgs &a, bool backward) {
        bytes = 0;
        const auto take = [&](size_t n) {
            const size_t at = bytes;
            bytes += (n + 255) & ~(size_t)255;
            return at;
        };
        pitch_d = (a.D + 7) / 8 * 8;
        pitch_f = (a.F + 7) / 8 * 8;
        pad = sizeof(T) == 2 && pitch_d != a.D;
        X = take(pad ? a.rows * pitch_d * sizeof(T) : 0);
        Wg = take(pad ? a.F * pitch_d * sizeof(T) : 0);
        Wu = take(pad ? a.F * pitch_d * sizeof(T) : 0);
        if (!backward) return;
        dG = take(a.rows * pitch_f * sizeof(T));
        dU = take(a.rows * pitch_f * sizeof(T));
        // whatever the alignment will be
        const int b1 = gated_grad_row_blocks(a.rows, a.F, 1);
        const int bv = gated_grad_row_blocks(a.rows, a.F, kVec<T>);
        partials = take((size_t)(b1 > bv ? b1 : bv) * 2 * a.F * sizeof(float));
    }
};

template <typename T> size_t gated_ws_bytes(const GatedArgs &a, bool backward) {
    return a.rows == 0 || a.F == 0 ? 0 : GatedLayout<T>(a, backward).bytes;
}

// X, Wg and Wu as TMA reads them: where they lie, or copied.
template <typename T>
cudaError_t gated_operands(const GatedArgs &a, const GatedPtrs &p, const GatedLayout<T> &at,
                           char *ws, GtMatrix (&m)[3], bool *launched, cudaStream_t s) {
    const void *from[3] = {p.X, p.Wg, p.Wu};
    const size_t to[3] = {at.X, at.Wg, at.Wu};
    for (int i = 0; i < 3; ++i) {
        const int64_t rows = i == 0 ? a.rows : a.F;
        m[i] = {from[i], rows, a.D, at.pitch_d};
        if (!at.pad) continue;
        m[i].at = ws + to[i];
        const int64_t n = rows * a.D, blocks = (n + 1023) / 1024;
        gated_pad_kernel<T><<<(unsigned)(blocks < 8 * kGatedSms ? blocks : 8 * kGatedSms), 256, 0, s>>>(
            (const T *)from[i], (T *)(ws + to[i]), n, a.D, at.pitch_d);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        *launched = true;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_gated(const GatedArgs &a, const GatedPtrs &p, void *ws, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        GtMatrix m[3];
        bool used = false, launched = false;
        cudaError_t e = gated_operands(a, p, GatedLayout<T>(a, false), (char *)ws, m, &launched, s);
        if (e == cudaSuccess)
            e = launch_gt_forward<T>(a, p, m[0], m[1], m[2], launched, s, &used);
        if (e != cudaSuccess || used) return e;
    }
    gated_simt_kernel<T><<<(unsigned)simt_blocks(a.rows, a.F), kSimtThreads, 0, s>>>(a, p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gated_backward(const GatedArgs &a, const GatedPtrs &p, void *ws,
                                  cudaStream_t s) {
    const GatedLayout<T> at(a, true);
    char *base = (char *)ws;
    T *dG = (T *)(base + at.dG), *dU = (T *)(base + at.dU);
    float *partials = (float *)(base + at.partials);
    const bool wide = a.F % kVec<T> == 0 && aligned16(p.dH) && aligned16(p.G) && aligned16(p.U);
    GtMatrix m[3];
    bool launched = false;
    cudaError_t e = cudaSuccess;
    if (sizeof(T) == 2) e = gated_operands(a, p, at, base, m, &launched, s);
    if (e != cudaSuccess) return e;
    e = wide ? launch_gated_grad<T, kVec<T>>(a, p, dG, dU, at.pitch_f, partials, s)
             : launch_gated_grad<T, 1>(a, p, dG, dU, at.pitch_f, partials, s);
    if (e != cudaSuccess) return e;
    if (p.dbg) {
        const int blocks = gated_grad_row_blocks(a.rows, a.F, wide ? kVec<T> : 1);
        e = launch_gated_bias_sums<T>(a, p, partials, blocks, true, s);
        if (e != cudaSuccess) return e;
    }
    if constexpr (sizeof(T) == 2) {
        bool used = false;
        e = launch_gt_backward<T>(a, p, m[0], m[1], m[2], {dG, a.rows, a.F, at.pitch_f},
                                  {dU, a.rows, a.F, at.pitch_f}, true, s, &used);
        if (e != cudaSuccess || used) return e;
    }
    const auto product = [&](SimtProduct q, void *out) {
        return launch_next(true, gated_simt_product_kernel<T>, dim3((unsigned)simt_blocks(q.M, q.N)),
                           kSimtThreads, 0, s, q, (T *)out);
    };
    e = product({{dG, dU}, {p.Wg, p.Wu}, at.pitch_f, 1, 1, a.D, a.rows, a.D, a.F, 2}, p.dX);
    if (e != cudaSuccess) return e;
    e = product({{dG, dG}, {p.X, p.X}, 1, at.pitch_f, 1, a.D, a.F, a.D, a.rows, 1}, p.dWg);
    if (e != cudaSuccess) return e;
    return product({{dU, dU}, {p.X, p.X}, 1, at.pitch_f, 1, a.D, a.F, a.D, a.rows, 1}, p.dWu);
}

#define GS_GATED_INST(T)                                                                         \
    template size_t gated_ws_bytes<T>(const GatedArgs &, bool);                                   \
    template cudaError_t launch_gated<T>(const GatedArgs &, const GatedPtrs &, void *,            \
                                         cudaStream_t);                                           \
    template cudaError_t launch_gated_backward<T>(const GatedArgs &, const GatedPtrs &, void *,   \
                                                  cudaStream_t);

}  // namespace gs
