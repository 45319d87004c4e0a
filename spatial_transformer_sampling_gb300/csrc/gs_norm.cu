// gs_norm.cu -- layer norm over the last axis, forward and backward.
//
// Forward, per row x of D elements (fp32 throughout, one rounding at the store):
//   mean = sum x / D, var = sum (x - mean)^2 / D, inv = 1 / sqrt(var + eps),
//   y = (x - mean) * inv * scale + B.
// Backward, with xhat = (x - mean) * inv and g = dy * scale:
//   dx = inv * (g - sum(g) / D - xhat * sum(g * xhat) / D),
//   dscale = sum over rows of dy * xhat,  dB = sum over rows of dy.
//
// Both read their inputs once: a row stays in the registers of the L threads
// that share it (8, 16, 32 or a block of 256), NV runs of V elements each, up
// to D = 8192; longer rows are read again for each pass.  The backward pass
// walks rows with a fixed set of blocks, so that a thread keeps the sums of its
// columns over all its rows; a second kernel adds the blocks in order.
#include "gs_internal.h"
#include "gs_ptx.cuh"
#include "gs_vec.cuh"

namespace gs {
namespace {

// Bound by memory.  16 x 256 x 256 rows of 64 fp32 forward: 91.4 us, 5.96 TB/s
// (0.88 of a copy's rate); 16384 x 1024 bf16 backward: 28.9 us with the sum over
// blocks, 3.5 TB/s (a row's two reductions stand between its loads and its store,
// and the sums that each block leaves behind are a tenth of the traffic).  Before
// the arithmetic was packed, a thread's scale kept and the blocks cut to what the
// registers hold at once, it took 41.9 us.
constexpr int kNormThreads = 256;
constexpr int kNormOnChip = 8192;      // widest row held in registers
constexpr int kNormSms = 152;

// Sum over the L threads of a row.  L = 256 uses shared memory, two slots in
// turn so that one barrier per sum suffices.
template <int L> __device__ __forceinline__ float row_sum(float v, int slot) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (L > 32) {
        __shared__ float s[2][L / 32 > 0 ? L / 32 : 1];
        if (threadIdx.x % 32 == 0) s[slot][threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < L / 32; ++w) v += s[slot][w];
    }
    return v;
}

// R rows per group of L threads, loads of all of them first.
template <typename T, int V, int L, int NV, int R>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_kernel(const T *X, const T *scale, const T *B, T *Y, float *mean, float *inv,
                      NormArgs a) {
    using IOV = Run<T, V>;
    constexpr int kGroups = kNormThreads / L;
    const int part = threadIdx.x % L;
    const int64_t row0 = ((int64_t)blockIdx.x * kGroups + threadIdx.x / L) * R;
    typename IOV::Raw raw[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            raw[r][k] = row0 + r < a.rows && d < a.D ? IOV::load(X + (row0 + r) * a.D + d) : IOV::zero();
        }
    float x[R][NV][V], m[R], iv[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            IOV::widen(raw[r][k], x[r][k]);
#pragma unroll
            for (int e = 0; e < V; ++e) s += x[r][k][e];
        }
        m[r] = row_sum<L>(s, 0) / (float)a.D;
        s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const bool on = (k * L + part) * V < a.D;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                x[r][k][e] -= m[r];
                if (on) s = fmaf(x[r][k][e], x[r][k][e], s);
            }
        }
        iv[r] = 1.0f / sqrtf(row_sum<L>(s, 1) / (float)a.D + a.eps);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int d = (k * L + part) * V;
        if (d >= a.D) continue;
        float g[V], b[V] = {};
        IOV::widen(IOV::load(scale + d), g);
        if (B) IOV::widen(IOV::load(B + d), b);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.rows) continue;
            float y[V];
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = fmaf(x[r][k][e] * iv[r], g[e], b[e]);
            IOV::store(Y + (row0 + r) * a.D + d, y);
        }
    }
    if (part == 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.rows) continue;
            if (mean) mean[row0 + r] = m[r];
            if (inv) inv[row0 + r] = iv[r];
        }
    }
}

// Rows wider than kNormOnChip: a block per row, three passes.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_wide_kernel(const T *X, const T *scale, const T *B, T *Y, float *mean, float *inv,
                           NormArgs a) {
    const int64_t row = blockIdx.x;
    const T *x = X + row * a.D;
    float s = 0.0f;
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) s += IO<T>::ld(x + d);
    const float m = row_sum<kNormThreads>(s, 0) / (float)a.D;
    s = 0.0f;
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        const float c = IO<T>::ld(x + d) - m;
        s = fmaf(c, c, s);
    }
    const float r = 1.0f / sqrtf(row_sum<kNormThreads>(s, 1) / (float)a.D + a.eps);
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        const float b = B ? IO<T>::ld(B + d) : 0.0f;
        Y[row * a.D + d] = IO<T>::st(fmaf((IO<T>::ld(x + d) - m) * r, IO<T>::ld(scale + d), b));
    }
    if (threadIdx.x == 0) {
        if (mean) mean[row] = m;
        if (inv) inv[row] = r;
    }
}

// Sums of two values over the L threads of a row; slots alternate between calls,
// so that one barrier per call suffices.
template <int L> __device__ __forceinline__ void row_sum2(float &a, float &b, int slot) {
    if (L < 32) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        return;
    }
    // the lower half of a warp goes on with a, the upper half with b
    const int lane = threadIdx.x % 32;
    float v = lane < 16 ? a : b;
    v += __shfl_xor_sync(0xffffffffu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (L == 32) {
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
    } else {
        constexpr int W = L > 32 ? L / 32 : 1;
        __shared__ float s[2][2][kNormThreads / 32];
        if (lane % 16 == 0) s[slot][lane / 16][threadIdx.x / 32] = v;
        __syncthreads();
        a = b = 0.0f;
        const int first = threadIdx.x / L * W;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += s[slot][0][first + w];
            b += s[slot][1][first + w];
        }
    }
}

// Blocks per SM of the backward pass, by the elements of a row that a thread holds.
constexpr int norm_backward_blocks(int N) { return N <= 4 ? 4 : N <= 8 ? 3 : N <= 16 ? 2 : 1; }

// dX of the block's rows and, into partials[block], its column sums (the sums
// for dScale, then those for dB).  The next row's loads are issued before this
// one is worked on.
template <typename T, int V, int L, int NV>
__global__ void __launch_bounds__(kNormThreads, norm_backward_blocks(NV * V))
    layer_norm_backward_kernel(const T *dY, const T *X, const T *scale, const float *mean,
                               const float *inv, T *dX, float *partials, NormArgs a) {
    using IOV = Run<T, V>;
    constexpr int kGroups = kNormThreads / L;
    constexpr int N = NV * V, P = (N + 1) / 2;   // a thread's elements, in pairs
    const int part = threadIdx.x % L, group = threadIdx.x / L;
    const float per_d = 1.0f / (float)a.D;
    float2 ds[P] = {}, db[P] = {};
    typename IOV::Raw rx[NV], rg[NV], rw[NV];
    float m = 0.0f, iv = 0.0f;
    // zeros behind a row's end, whose products and sums are zeros
    const auto load = [&](int64_t row) {
        const bool here = row < a.rows;
        const int64_t at = row * a.D;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = here && d < a.D;
            rx[k] = on ? IOV::load(X + at + d) : IOV::zero();
            rg[k] = on ? IOV::load(dY + at + d) : IOV::zero();
        }
        m = here ? __ldg(mean + row) : 0.0f;
        iv = here ? __ldg(inv + row) : 0.0f;
    };
    const auto load_scale = [&] {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            rw[k] = d < a.D ? IOV::load(scale + d) : IOV::zero();
        }
    };
    const auto pairs_of = [](const typename IOV::Raw (&r)[NV], float2 (&v)[P]) {
        float f[2 * P] = {};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float e[V];
            IOV::widen(r[k], e);
#pragma unroll
            for (int i = 0; i < V; ++i) f[k * V + i] = e[i];
        }
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = make_float2(f[2 * p], f[2 * p + 1]);
    };
    const auto element = [](const float2 (&v)[P], int i) { return i % 2 ? v[i / 2].y : v[i / 2].x; };
    const int64_t step = (int64_t)gridDim.x * kGroups;
    int64_t row = (int64_t)blockIdx.x * kGroups + group;
    load(row);
    if (NV == 1) load_scale();   // stays in registers
    int slot = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kGroups; row0 < a.rows; row0 += step, row += step) {
        float2 xh[P], gw[P], w[P], t0 = {}, t1 = {};
        if (NV > 1) load_scale();
        pairs_of(rx, xh);
        pairs_of(rg, gw);
        pairs_of(rw, w);
        const float2 minus_m = make_float2(-m, -m), iv2 = make_float2(iv, iv);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            xh[p] = mul_f32x2(add_f32x2(xh[p], minus_m), iv2);
            ds[p] = fma_f32x2(gw[p], xh[p], ds[p]);
            db[p] = add_f32x2(db[p], gw[p]);
            gw[p] = mul_f32x2(gw[p], w[p]);
            t0 = add_f32x2(t0, gw[p]);
            t1 = fma_f32x2(gw[p], xh[p], t1);
        }
        float s0 = t0.x + t0.y, s1 = t1.x + t1.y;
        if (isinf(m * iv)) {   // behind the row's end, 0 * ((0 - m) * iv) is no zero then
            s1 = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((i / V * L + part) * V < a.D)
                    s1 = fmaf(element(gw, i), element(xh, i), s1);
        }
        load(row + step);
        row_sum2<L>(s0, s1, slot);
        slot ^= 1;
        if (row >= a.rows) continue;
        s0 *= -per_d;
        s1 *= -per_d;
        float out[2 * P];
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float2 g0 = add_f32x2(gw[p], make_float2(s0, s0));
            const float2 v = mul_f32x2(fma_f32x2(xh[p], make_float2(s1, s1), g0), iv2);
            out[2 * p] = v.x;
            out[2 * p + 1] = v.y;
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            float e[V];
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = out[k * V + i];
            if (d < a.D) IOV::store(dX + row * a.D + d, e);
        }
    }
    if (!partials) return;
    // the groups of the block in order; one column run of every thread at a time
    float *out = partials + (int64_t)blockIdx.x * 2 * a.D;
    __shared__ float s_ds[kNormThreads * V], s_db[kNormThreads * V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        if (kGroups > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s_ds[threadIdx.x * V + e] = element(ds, k * V + e);
                s_db[threadIdx.x * V + e] = element(db, k * V + e);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < L * V; c += kNormThreads) {
                const int d = k * L * V + c;
                float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    t0 += s_ds[g * L * V + c];
                    t1 += s_db[g * L * V + c];
                }
                if (d < a.D) {
                    out[d] = t0;
                    out[a.D + d] = t1;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int d = (k * L + part) * V + e;
                if (d < a.D) {
                    out[d] = element(ds, k * V + e);
                    out[a.D + d] = element(db, k * V + e);
                }
            }
        }
    }
}

// Rows wider than kNormOnChip: a block per row for dX, then a thread per column
// for the sums of a block of rows.
template <typename T>
__global__ void __launch_bounds__(kNormThreads)
    layer_norm_wide_dx_kernel(const T *dY, const T *X, const T *scale, const float *mean,
                              const float *inv, T *dX, NormArgs a) {
    const int64_t row = blockIdx.x;
    const T *x = X + row * a.D, *dy = dY + row * a.D;
    const float m = mean[row], r = inv[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        const float g = IO<T>::ld(dy + d) * IO<T>::ld(scale + d);
        s0 += g;
        s1 = fmaf(g, (IO<T>::ld(x + d) - m) * r, s1);
    }
    s0 = row_sum<kNormThreads>(s0, 0) / (float)a.D;
    s1 = row_sum<kNormThreads>(s1, 1) / (float)a.D;
    for (int d = threadIdx.x; d < a.D; d += kNormThreads) {
        const float g = IO<T>::ld(dy + d) * IO<T>::ld(scale + d);
        dX[row * a.D + d] = IO<T>::st(r * (g - s0 - (IO<T>::ld(x + d) - m) * r * s1));
    }
}
template <typename T>
__global__ void layer_norm_wide_partial_kernel(const T *dY, const T *X, const float *mean,
                                               const float *inv, float *partials, NormArgs a) {
    const int d = blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= a.D) return;
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
        const float g = IO<T>::ld(dY + row * a.D + d);
        s0 = fmaf(g, (IO<T>::ld(X + row * a.D + d) - mean[row]) * inv[row], s0);
        s1 += g;
    }
    partials[(int64_t)blockIdx.y * 2 * a.D + d] = s0;
    partials[((int64_t)blockIdx.y * 2 + 1) * a.D + d] = s1;
}

// dScale (y = 0) and dB (y = 1) from the blocks' sums: 32 columns a block, 32
// threads per column with every 32nd block each, joined in order.
template <typename T>
__global__ void __launch_bounds__(1024)
    layer_norm_finish_kernel(const float *partials, int blocks, T *dScale, T *dB, int D) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32, d = blockIdx.x * 32 + lane;
    T *out = blockIdx.y ? dB : dScale;
    if (!out) return;
    float sum = 0.0f;
    wait_for_previous_kernel(partials);
#pragma unroll 8
    for (int b = slice; b < blocks; b += 32)
        if (d < D) sum += __ldg(partials + ((int64_t)b * 2 + blockIdx.y) * D + d);
    s[slice][lane] = sum;
    __syncthreads();
    // a warp per column: lane `lane` holds slice `lane` of column `slice`
    float v = s[lane][slice];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 32 + slice < D) out[blockIdx.x * 32 + slice] = IO<T>::st(v);
}

// Calls f(L, NV) with the threads per row and the runs per thread for a row of
// `runs` runs: a warp or less while a thread's share is small (no barrier in
// its sums), a block beyond that.
template <int V, typename F> cudaError_t norm_shape(int runs, F &&f) {
    using std::integral_constant;
    if (runs <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (runs <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (runs <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (runs <= 64) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
    if (runs <= 128) return f(integral_constant<int, 32>(), integral_constant<int, 4>());
    if (runs <= 256 && V > 1) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (runs <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 8>());
    if (runs <= 512 && V > 1) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (runs <= 1024) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    if constexpr (V <= 4)
        if (runs <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 8>());
    if constexpr (V == 1)
        return runs <= 4096 ? f(integral_constant<int, 256>(), integral_constant<int, 16>())
                            : f(integral_constant<int, 256>(), integral_constant<int, 32>());
    return cudaErrorInvalidValue;   // not reached: D <= kNormOnChip
}

// Calls f(L, NV) for the backward pass: as many threads per row as keep a
// thread's share, and with it the sums it holds, to one run (a block of 256 at
// most: of 1024, with fewer blocks per SM to wait for each other's barriers, 8192
// x 4096 fp32 takes 78.8 us instead of 68.2), so that many warps share an SM.
template <int V, typename F> cudaError_t norm_backward_shape(int runs, F &&f) {
    using std::integral_constant;
    if (runs <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (runs <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (runs <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (runs <= 64) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (runs <= 128) return f(integral_constant<int, 128>(), integral_constant<int, 1>());
    if (runs <= 256) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (runs <= 512) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (runs <= 1024) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    if constexpr (V <= 4)
        if (runs <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 8>());
    if constexpr (V == 1)
        return runs <= 4096 ? f(integral_constant<int, 256>(), integral_constant<int, 16>())
                            : f(integral_constant<int, 256>(), integral_constant<int, 32>());
    return cudaErrorInvalidValue;   // not reached: D <= kNormOnChip
}

// Row blocks of the backward pass: what an SM holds of them at once, and no
// more, since each leaves 2 D sums behind.
int row_blocks(int64_t rows, int L, int per_sm) {
    const int64_t b = (rows + kNormThreads / L - 1) / (kNormThreads / L);
    const int most = kNormSms * per_sm;
    return (int)(b < most ? b : most);
}
constexpr int kWideBlocks = 2;   // of rows, per SM, for rows wider than kNormOnChip
template <int V> int row_blocks_of(int64_t rows, int64_t D) {
    int blocks = row_blocks(rows, kNormThreads, kWideBlocks);
    if (D <= kNormOnChip)
        norm_backward_shape<V>((int)((D + V - 1) / V), [&](auto l, auto nv) {
            blocks = row_blocks(rows, decltype(l)::value, norm_backward_blocks(V * decltype(nv)::value));
            return cudaSuccess;
        });
    return blocks;
}

template <typename T, int V>
cudaError_t run_forward(const T *X, const T *scale, const T *B, T *Y, float *mean, float *inv,
                        const NormArgs &a, cudaStream_t s) {
    return norm_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        constexpr int R = L == 256 || NV > 2 ? 1 : NV == 2 ? 2 : 4;   // about four runs in flight
        constexpr int kRows = kNormThreads / L * R;
        layer_norm_kernel<T, V, L, NV, R>
            <<<(unsigned)((a.rows + kRows - 1) / kRows), kNormThreads, 0, s>>>(X, scale, B, Y, mean,
                                                                              inv, a);
        return cudaGetLastError();
    });
}

template <typename T, int V>
cudaError_t run_backward(const T *dY, const T *X, const T *scale, const float *mean,
                         const float *inv, T *dX, float *partials, int *blocks, const NormArgs &a,
                         cudaStream_t s) {
    return norm_backward_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        *blocks = row_blocks(a.rows, L, norm_backward_blocks(NV * V));
        layer_norm_backward_kernel<T, V, L, NV>
            <<<*blocks, kNormThreads, 0, s>>>(dY, X, scale, mean, inv, dX, partials, a);
        return cudaGetLastError();
    });
}

}  // namespace

int layer_norm_partial_blocks(int64_t rows, int64_t D) {
    // whatever the type and alignment will be
    const int b1 = row_blocks_of<1>(rows, D), b4 = row_blocks_of<4>(rows, D);
    const int b8 = row_blocks_of<8>(rows, D);
    return b1 > b4 ? (b1 > b8 ? b1 : b8) : (b4 > b8 ? b4 : b8);
}

template <typename T>
cudaError_t launch_layer_norm(const void *X, const void *scale, const void *B, void *Y, float *mean,
                              float *inv, const NormArgs &a, cudaStream_t s) {
    const T *x = (const T *)X, *g = (const T *)scale, *b = (const T *)B;
    if (a.D > kNormOnChip) {
        layer_norm_wide_kernel<T><<<(unsigned)a.rows, kNormThreads, 0, s>>>(x, g, b, (T *)Y, mean, inv, a);
        return cudaGetLastError();
    }
    if (a.D % kVec<T> == 0 && aligned16(X) && aligned16(scale) && aligned16(B) && aligned16(Y))
        return run_forward<T, kVec<T>>(x, g, b, (T *)Y, mean, inv, a, s);
    return run_forward<T, 1>(x, g, b, (T *)Y, mean, inv, a, s);
}

template <typename T>
cudaError_t launch_layer_norm_backward(const void *dY, const void *X, const void *scale,
                                       const float *mean, const float *inv, void *dX, void *dScale,
                                       void *dB, float *partials, const NormArgs &a,
                                       cudaStream_t s) {
    const T *dy = (const T *)dY, *x = (const T *)X, *g = (const T *)scale;
    float *sums = dScale || dB ? partials : nullptr;
    int blocks = 0;
    cudaError_t e = cudaSuccess;
    if (a.rows > 0 && a.D > kNormOnChip) {
        layer_norm_wide_dx_kernel<T>
            <<<(unsigned)a.rows, kNormThreads, 0, s>>>(dy, x, g, mean, inv, (T *)dX, a);
        blocks = row_blocks(a.rows, kNormThreads, kWideBlocks);
        if (sums)
            layer_norm_wide_partial_kernel<T>
                <<<dim3((a.D + 255) / 256, blocks), 256, 0, s>>>(dy, x, mean, inv, sums, a);
        e = cudaGetLastError();
    } else if (a.rows > 0) {
        if (a.D % kVec<T> == 0 && aligned16(dY) && aligned16(X) && aligned16(scale) && aligned16(dX))
            e = run_backward<T, kVec<T>>(dy, x, g, mean, inv, (T *)dX, sums, &blocks, a, s);
        else
            e = run_backward<T, 1>(dy, x, g, mean, inv, (T *)dX, sums, &blocks, a, s);
    }
    if (e != cudaSuccess || !(dScale || dB)) return e;
    return launch_next(blocks > 0, layer_norm_finish_kernel<T>, dim3((a.D + 31) / 32, 2), 1024, 0, s,
                       partials, blocks, (T *)dScale, (T *)dB, a.D);
}

#define GS_NORM_INST(T)                                                                           \
    template cudaError_t launch_layer_norm<T>(const void *, const void *, const void *, void *,   \
                                              float *, float *, const NormArgs &, cudaStream_t);  \
    template cudaError_t launch_layer_norm_backward<T>(                                           \
        const void *, const void *, const void *, const float *, const float *, void *, void *,   \
        void *, float *, const NormArgs &, cudaStream_t);
GS_NORM_INST(float)
GS_NORM_INST(__half)
GS_NORM_INST(__nv_bfloat16)
#undef GS_NORM_INST

}  // namespace gs
