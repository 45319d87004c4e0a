// gs_gated_launch.cuh -- workspace layout and launches of the gated projections.
#pragma once

#include "gs_gated_few.cuh"
#include "gs_gated_grad.cuh"
#include "gs_gated_simt.cuh"
#include "gs_gated_tc.cuh"

namespace gs {

// Rows of up to three matrices copied to a pitch of whole 16-byte runs, fp32 as planes
// rows * pitch elements apart; what lies behind a row's end is not written (and not
// read: the tensor maps end with the row).
template <typename T> struct PadArgs {
    const T *from[3];
    Factor<T> *to[3];
    int64_t rows[3];
    int width;
    int64_t pitch;
};
// A row is copied by `team` lanes, 8, 16 or 32; a run behind its end is copied too (the
// pitch is a multiple of one).
template <typename T, int READ>
__global__ void __launch_bounds__(256) gated_pad_kernel(PadArgs<T> p, int team) {
    constexpr int V = kRowsV<T, READ>;
    const int m = blockIdx.y, lane = threadIdx.x % team, per = 256 / team;
    // chosen here: an index into the arguments would copy them to the stack
    const int64_t rows = m == 0 ? p.rows[0] : m == 1 ? p.rows[1] : p.rows[2], total = rows * p.width;
    const T *from = m == 0 ? p.from[0] : m == 1 ? p.from[1] : p.from[2];
    Factor<T> *all = m == 0 ? p.to[0] : m == 1 ? p.to[1] : p.to[2];
    for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / team; r < rows; r += (int64_t)gridDim.x * per) {
        const int64_t at = r * p.width;
        Factor<T> *to = all + r * p.pitch;
#pragma unroll 4
        for (int d = lane * V; d < p.width; d += team * V) {
            const auto run = row_load<T, READ>(from, at + d, total);
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<std::remove_const_t<decltype(run)> *>(to + d) = run;
            } else {
                float v[V];
                Run<T, V>::widen(run, v);
                store_factor<T, V>(to + d, rows * p.pitch, v);
            }
        }
    }
}

// Workspace: copies of X, Wg and Wu where rows are no multiple of 16 bytes, or their
// planes; backward, dG and dU, the biases' partial sums and those of shared products.
template <typename T> struct GatedLayout {
    int64_t pitch_d, pitch_f;
    bool copy;
    size_t X, Wg, Wu, dG, dU, partials, sums, bound, bytes;
    GatedLayout(const GatedArgs &a, bool backward) {
        bytes = 0;
        const auto take = [&](int64_t n) {
            const size_t at = bytes;
            bytes += ((size_t)n + 255) & ~(size_t)255;
            return at;
        };
        const int each = sizeof(T) == 4 ? 6 : 2;   // bytes of an element in its planes
        pitch_d = (a.D + 7) / 8 * 8;
        pitch_f = (a.F + 7) / 8 * 8;
        copy = sizeof(T) == 4 || pitch_d != a.D;
        X = take(copy ? a.rows * pitch_d * each : 0);
        Wg = take(copy ? a.F * pitch_d * each : 0);
        Wu = take(copy ? a.F * pitch_d * each : 0);
        if (!backward) return;
        dG = take(a.rows * pitch_f * each);
        dU = take(a.rows * pitch_f * each);
        // whatever the alignment will be
        const int b1 = grad_plan(a.rows, a.F, 1).rows;
        const int bv = grad_plan(a.rows, a.F, kVec<T>).rows;
        partials = take((int64_t)(b1 > bv ? b1 : bv) * 2 * a.F * sizeof(float));
        sums = take(gt_backward_plan<T>(a).bytes());
        bound = take(__is_same(T, __half) ? sizeof(uint32_t) : 0);
    }
};

template <typename T> size_t gated_ws_bytes(const GatedArgs &a, bool backward) {
    if (a.rows == 0 || a.F == 0 || (!backward && gated_few_takes<T>(a))) return 0;
    return GatedLayout<T>(a, backward).bytes;
}

// X, Wg and Wu as TMA reads them: where they lie, or copied.
template <typename T>
cudaError_t gated_operands(const GatedArgs &a, const GatedPtrs &p, const GatedLayout<T> &at,
                           char *ws, GtMatrix (&m)[3], cudaStream_t s) {
    const void *from[3] = {p.X, p.Wg, p.Wu};
    const size_t to[3] = {at.X, at.Wg, at.Wu};
    PadArgs<T> q;
    q.width = a.D;
    q.pitch = at.pitch_d;
    const int read = rows_read<T>(a.D, {p.X, p.Wg, p.Wu});
    for (int i = 0; i < 3; ++i) {
        q.rows[i] = i == 0 ? a.rows : a.F;
        q.from[i] = (const T *)from[i];
        q.to[i] = (Factor<T> *)(ws + to[i]);
        m[i] = {at.copy ? (const void *)q.to[i] : from[i], q.rows[i], a.D, at.pitch_d};
    }
    if (!at.copy) return cudaSuccess;
    const int runs = (a.D + kVec<T> - 1) / kVec<T>, team = runs <= 8 ? 8 : runs <= 16 ? 16 : 32;
    const int64_t need = ((a.rows > a.F ? a.rows : a.F) * team + 255) / 256;
    const dim3 grid((unsigned)(need < 8 * kGatedSms ? need : 8 * kGatedSms), 3);
    auto kernel = read == kRowsSingle ? gated_pad_kernel<T, kRowsSingle> : gated_pad_kernel<T, kRowsShifted>;
    if constexpr (sizeof(T) == 4) {   // 16-bit rows of whole runs are read where they lie
        if (read == kRowsRuns) kernel = gated_pad_kernel<T, kRowsRuns>;
    }
    kernel<<<grid, 256, 0, s>>>(q, team);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gated(const GatedArgs &a, const GatedPtrs &p, void *ws, cudaStream_t s) {
    if (gated_few_takes<T>(a)) return launch_gated_few<T>(a, p, s);
    if (gt_forward_takes<T>(a)) {   // longer rows are read where they lie, not copied
        GtMatrix m[3];
        const GatedLayout<T> at(a, false);
        bool used = false;
        cudaError_t e = gated_operands(a, p, at, (char *)ws, m, s);
        if (e == cudaSuccess) e = launch_gt_forward<T>(a, p, m[0], m[1], m[2], at.copy, s, &used);
        if (e != cudaSuccess || used) return e;
    }
    if constexpr (sizeof(T) == 2) {
        gated_simt_kernel<T><<<(unsigned)simt_blocks(a.rows, a.F), kSimtThreads, 0, s>>>(a, p);
        return cudaGetLastError();
    }
    return cudaErrorInvalidValue;   // not reached: planes are 16-byte aligned
}

template <typename T>
cudaError_t launch_gated_backward(const GatedArgs &a, const GatedPtrs &p, void *ws,
                                  cudaStream_t s) {
    const GatedLayout<T> at(a, true);
    char *base = (char *)ws;
    Factor<T> *dG = (Factor<T> *)(base + at.dG), *dU = (Factor<T> *)(base + at.dU);
    float *partials = (float *)(base + at.partials);
    const int read = rows_read<T>(a.F, {p.dH, p.G, p.U});
    GtMatrix m[3];
    cudaError_t e = gated_operands(a, p, at, base, m, s);
    if (e != cudaSuccess) return e;
    uint32_t *bound = (uint32_t *)(base + at.bound);
    if constexpr (__is_same(T, __half)) {
        e = launch_gated_bound<T>(a, p, read != kRowsSingle, bound, s);
        if (e != cudaSuccess) return e;
    }
    e = read == kRowsSingle ? launch_gated_grad<T, kRowsSingle>(a, p, dG, dU, at.pitch_f, partials, bound, s)
        : read == kRowsRuns ? launch_gated_grad<T, kRowsRuns>(a, p, dG, dU, at.pitch_f, partials, bound, s)
                            : launch_gated_grad<T, kRowsShifted>(a, p, dG, dU, at.pitch_f, partials, bound, s);
    if (e != cudaSuccess) return e;
    if (p.dbg) {
        const int blocks = grad_plan(a.rows, a.F, read == kRowsSingle ? 1 : kVec<T>).rows;
        e = launch_gated_bias_sums<T>(a, p, partials, blocks, true, s);
        if (e != cudaSuccess) return e;
    }
    bool used = false;
    e = launch_gt_backward<T>(a, p, m[0], m[1], m[2], {dG, a.rows, a.F, at.pitch_f},
                              {dU, a.rows, a.F, at.pitch_f}, bound, (float *)(base + at.sums),
                              true, s, &used);
    if (e != cudaSuccess || used) return e;
    if constexpr (sizeof(T) == 2) {
        const auto product = [&](SimtProduct q, void *out) {
            return launch_next(true, gated_simt_product_kernel<T>,
                               dim3((unsigned)simt_blocks(q.M, q.N)), kSimtThreads, 0, s, q, (T *)out);
        };
        e = product({{dG, dU}, {p.Wg, p.Wu}, at.pitch_f, 1, 1, a.D, a.rows, a.D, a.F, 2, bound}, p.dX);
        if (e != cudaSuccess) return e;
        e = product({{dG, dG}, {p.X, p.X}, 1, at.pitch_f, 1, a.D, a.F, a.D, a.rows, 1, bound}, p.dWg);
        if (e != cudaSuccess) return e;
        return product({{dU, dU}, {p.X, p.X}, 1, at.pitch_f, 1, a.D, a.F, a.D, a.rows, 1, bound}, p.dWu);
    }
    return cudaErrorInvalidValue;   // not reached: planes are 16-byte aligned
}

#define GS_GATED_INST(T)                                                                         \
    template size_t gated_ws_bytes<T>(const GatedArgs &, bool);                                   \
    template cudaError_t launch_gated<T>(const GatedArgs &, const GatedPtrs &, void *,            \
                                         cudaStream_t);                                           \
    template cudaError_t launch_gated_backward<T>(const GatedArgs &, const GatedPtrs &, void *,   \
                                                  cudaStream_t);

}  // namespace gs
