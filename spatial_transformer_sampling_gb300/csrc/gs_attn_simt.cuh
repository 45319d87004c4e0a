// gs_attn_simt.cuh -- attention forward and backward in fp32 arithmetic, for
// fp32 tensors and for 16-bit ones whose rows the tensor-core kernels cannot
// take (head widths or strides that are not multiples of 16 bytes).
//
// 64 x 64 score tiles, 256 threads, 4 x 4 values each, every product as a
// register-tiled outer product over operands in shared memory laid out
// contraction-major ([k][64 + 4]): per step two 16-byte shared loads feed
// eight packed FMAs.  Rows (queries; keys in the dK / dV kernel) stay resident,
// columns are walked tile by tile; weights and their gradients go back through
// shared memory, over the columns' transposed copy, as the first operand of the
// next product.  One block sums each gradient in one order.
#pragma once

#include "gs_attn_common.cuh"
#include "gs_attn_rel.cuh"
#include "gs_ptx.cuh"
#include "gs_vec.cuh"

namespace gs {

constexpr int kSimtTile = 64;
constexpr int kSimtThreads = 256;
constexpr int kSimtPitch = kSimtTile + 4;   // keeps 16-byte alignment, spreads banks

// Element offsets of one operand: base + n, h, token strides.
template <typename T> struct SimtView {
    const T *p;
    int64_t by_token;
    __device__ __forceinline__ SimtView(const void *base, const int64_t (&s)[3], int n, int h)
        : p((const T *)base + n * s[0] + h * s[2]), by_token(s[1]) {}
};

// dst[d][64] from 64 tokens, zeros from `live` on; a thread reads along a row,
// V elements at a time (16 bytes, or one where rows are not aligned).
template <typename T, int V>
__device__ __forceinline__ void simt_load_t(float *dst, const SimtView<T> &v, int row0, int live,
                                            int D) {
    const int row = threadIdx.x % kSimtTile;
    const T *p = v.p + (int64_t)(row0 + row) * v.by_token;
    const bool on = row < live;
#pragma unroll 4
    for (int d = threadIdx.x / kSimtTile * V; d < D; d += kSimtThreads / kSimtTile * V) {
        float x[V] = {};
        if (on) Run<T, V>::widen(Run<T, V>::load(p + d), x);
#pragma unroll
        for (int e = 0; e < V; ++e) dst[(d + e) * kSimtPitch + row] = x[e];
    }
}

// dst[64][pitch] (D values a row) from 64 tokens, zeros from `live` on and
// behind a row.
template <typename T, int V>
__device__ __forceinline__ void simt_load_n(float *dst, int pitch, const SimtView<T> &v, int row0,
                                            int live, int D) {
    const int runs = (pitch + V - 1) / V;
#pragma unroll 4
    for (int k = threadIdx.x; k < kSimtTile * runs; k += kSimtThreads) {
        const int row = k / runs, d = (k - row * runs) * V;
        float x[V] = {};
        if (row < live && d < D)
            Run<T, V>::widen(Run<T, V>::load(v.p + (int64_t)(row0 + row) * v.by_token + d), x);
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (d + e < pitch) dst[row * pitch + d + e] = x[e];
    }
}

// c[4][4] += sum_k a[k][4 rows] b[k][4 columns]
__device__ __forceinline__ void simt_product(float2 (&c)[4][2], const float *a, int pitch_a,
                                             const float *b, int pitch_b, int K) {
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        const float4 x = *reinterpret_cast<const float4 *>(a + k * pitch_a);
        const float4 y = *reinterpret_cast<const float4 *>(b + k * pitch_b);
        const float2 y0 = make_float2(y.x, y.y), y1 = make_float2(y.z, y.w);
        const float r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            c[i][0] = fma_f32x2(make_float2(r[i], r[i]), y0, c[i][0]);
            c[i][1] = fma_f32x2(make_float2(r[i], r[i]), y1, c[i][1]);
        }
    }
}

__device__ __forceinline__ float &at(float2 (&c)[4][2], int i, int j) {
    return j % 2 ? c[i][j / 2].y : c[i][j / 2].x;
}

// Stores the transpose of the block's 64 x 64 tile: dst[column][row].
__device__ __forceinline__ void simt_store_t(float *dst, float2 (&c)[4][2], int ty, int tx) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(dst + (tx * 4 + j) * kSimtPitch + ty * 4) =
            make_float4(at(c, 0, j), at(c, 1, j), at(c, 2, j), at(c, 3, j));
}

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__host__ __device__ inline int simt_pitch_n(int D) { return (D + 3) / 4 * 4 + 4; }
// A transposed operand; one that weights are written over holds 64 rows at least.
__host__ __device__ inline int simt_floats_t(int D, bool reused) {
    return (reused && D < kSimtTile ? kSimtTile : D) * kSimtPitch;
}
inline int simt_fwd_smem(int D) {
    return (simt_floats_t(D, false) + simt_floats_t(D, true) + kSimtTile * simt_pitch_n(D)) * 4;
}
inline int simt_bwd_smem(int D, bool dkv, int rel) {
    return (2 * simt_floats_t(D, false) + 2 * simt_floats_t(D, true) +
            (dkv ? 2 : 1) * kSimtTile * simt_pitch_n(D)) * 4 + rel_smem(rel, 2);
}

// NC: 64-column chunks of the head width.
template <typename T, int NC, int E>
__global__ void __launch_bounds__(kSimtThreads)
    attn_simt_fwd_kernel(AttnArgs a, AttnPtrs p, const float *bias) {
    extern __shared__ float4 simt_smem[];
    const int D = a.D, pitch_n = simt_pitch_n(D);
    float *qt = reinterpret_cast<float *>(simt_smem), *kt = qt + simt_floats_t(D, false);
    float *vn = kt + simt_floats_t(D, true);
    const int tiles = (a.Lq + kSimtTile - 1) / kSimtTile;
    const int i0 = (int)(blockIdx.x % tiles) * kSimtTile;
    const int h = (int)(blockIdx.x / tiles % a.H), n = (int)(blockIdx.x / tiles / a.H);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    const float c2 = a.scale * kLog2e;
    const SimtView<T> Q(p.Q, a.qs, n, h), K(p.K, a.ks, n, h), V(p.V, a.vs, n, h);
    const int keys = keys_of(a, n);
    if (bias) bias += (int64_t)h * a.bias_stride;

    simt_load_t<T, E>(qt, Q, i0, a.Lq - i0, D);
    float2 o[NC][4][2] = {};
    float m[4], l[4];
    int rq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
        rq[i] = bias ? rel_q(a, min(i0 + ty * 4 + i, a.Lq - 1)) : 0;
    }
    for (int j0 = 0; j0 < keys; j0 += kSimtTile) {
        const int live = keys - j0;
        __syncthreads();
        simt_load_t<T, E>(kt, K, j0, live, D);
        simt_load_n<T, E>(vn, pitch_n, V, j0, live, D);
        __syncthreads();
        float2 s[4][2] = {};
        simt_product(s, qt + ty * 4, kSimtPitch, kt + tx * 4, kSimtPitch, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = tx * 4 + j < live;
            const int rk = bias && on ? rel_k(a, j0 + tx * 4 + j) : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float b = bias && on ? __ldg(bias + rq[i] - rk) : 0.0f;
                at(s, i, j) = on ? fmaf(at(s, i, j), c2, b) : -INFINITY;
            }
        }
        float keep[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float top = half_warp_max(fmaxf(
                m[i], fmaxf(fmaxf(at(s, i, 0), at(s, i, 1)), fmaxf(at(s, i, 2), at(s, i, 3)))));
            const float ref = top == -INFINITY ? 0.0f : top;   // no key yet: weights 0
            keep[i] = exp2_approx(m[i] - ref);
            m[i] = top;
            l[i] *= keep[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                at(s, i, j) = exp2_approx(at(s, i, j) - ref);
                l[i] += at(s, i, j);
            }
        }
        __syncthreads();
        simt_store_t(kt, s, ty, tx);
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[c][i][0] = mul_f32x2(o[c][i][0], make_float2(keep[i], keep[i]));
                o[c][i][1] = mul_f32x2(o[c][i][1], make_float2(keep[i], keep[i]));
            }
            if (c * 64 + tx * 4 < D)
                simt_product(o[c], kt + ty * 4, kSimtPitch, vn + c * 64 + tx * 4, pitch_n,
                             min(live, kSimtTile));
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float sum = half_warp_sum(l[i]), f = sum != 0.0f ? 1.0f / sum : 0.0f;
        const int row = i0 + ty * 4 + i;
        if (row >= a.Lq) continue;
        T *out = (T *)p.O + (((int64_t)n * a.Lq + row) * a.H + h) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c * 64 + tx * 4 + j < D)
                    out[c * 64 + tx * 4 + j] = IO<T>::st(at(o[c], i, j) * f);
        if (tx == 0 && p.lse)
            p.lse[((int64_t)n * a.H + h) * a.Lq + row] =
                sum != 0.0f ? (m[i] + log2f(sum)) * kLn2 : -INFINITY;
    }
}

// DKV: rows are keys, columns queries (dK, dV); else rows are queries, columns
// keys (dQ, and the bias gradient through `rel`, see RelWindow).
template <typename T, int NC, int E, bool DKV>
__device__ __forceinline__ void attn_simt_bwd_block(const AttnArgs &a, const AttnPtrs &p,
                                                    const float *bias, const float *lse2,
                                                    const float *delta, const RelArgs &rel,
                                                    int block) {
    extern __shared__ float4 simt_smem[];
    const int D = a.D, pitch_n = simt_pitch_n(D);
    float *r1 = reinterpret_cast<float *>(simt_smem), *r2 = r1 + simt_floats_t(D, false);
    float *t1 = r2 + simt_floats_t(D, false), *t2 = t1 + simt_floats_t(D, true);
    float *n1 = t2 + simt_floats_t(D, true), *n2 = n1 + kSimtTile * pitch_n;
    float *win_smem = DKV ? nullptr : n2;
    const int rows = DKV ? a.Lk : a.Lq;
    const int tiles = (rows + kSimtTile - 1) / kSimtTile;
    const int i0 = block % tiles * kSimtTile;
    const int nh = rel.head0 + block / tiles, h = nh % a.H, n = nh / a.H;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, warp = threadIdx.x / 32;
    const float c2 = a.scale * kLog2e;
    const int64_t dense[3] = {(int64_t)a.Lq * a.H * D, (int64_t)a.H * D, D};
    const SimtView<T> Q(p.Q, a.qs, n, h), K(p.K, a.ks, n, h), V(p.V, a.vs, n, h), G(p.dO, dense, n, h);
    const SimtView<T> &R1 = DKV ? K : Q, &R2 = DKV ? V : G, &C1 = DKV ? Q : K, &C2 = DKV ? G : V;
    const int keys = keys_of(a, n);
    const int live_rows = DKV ? keys : a.Lq;
    const int cols = i0 < live_rows ? (DKV ? a.Lq : keys) : 0;
    lse2 += (int64_t)nh * rows64(a.Lq);
    delta += (int64_t)nh * rows64(a.Lq);
    if (bias) bias += (int64_t)h * a.bias_stride;

    simt_load_t<T, E>(r1, R1, i0, live_rows - i0, D);
    simt_load_t<T, E>(r2, R2, i0, live_rows - i0, D);
    float2 acc1[NC][4][2] = {}, acc2[NC][4][2] = {};
    float row_lse[4], row_delta[4];
    int row_rel[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = min(i0 + ty * 4 + i, max(live_rows - 1, 0));
        row_lse[i] = DKV ? 0.0f : lse2[row];
        row_delta[i] = DKV ? 0.0f : delta[row];
        row_rel[i] = !bias ? 0 : DKV ? -rel_k(a, row) : rel_q(a, row);
    }
    // four warps, two per 32 queries, see to the bias gradient
    const bool with_rel = !DKV && rel.window > 0 && warp < 4 && i0 + warp / 2 * 32 < a.Lq && cols > 0;
    RelWindow win;
    float *rel_out = nullptr;
    if (with_rel) rel_out = win.init(a, win_smem, rel, i0, nh, warp / 2, warp % 2);

    for (int j0 = 0; j0 < cols; j0 += kSimtTile) {
        const int live = cols - j0;
        __syncthreads();
        simt_load_t<T, E>(t1, C1, j0, live, D);
        simt_load_t<T, E>(t2, C2, j0, live, D);
        simt_load_n<T, E>(n1, pitch_n, C1, j0, live, D);
        if (DKV) simt_load_n<T, E>(n2, pitch_n, C2, j0, live, D);
        __syncthreads();
        float2 s[4][2] = {}, d[4][2] = {};
        simt_product(s, r1 + ty * 4, kSimtPitch, t1 + tx * 4, kSimtPitch, D);
        simt_product(d, r2 + ty * 4, kSimtPitch, t2 + tx * 4, kSimtPitch, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = j0 + tx * 4 + j;
            const bool on = tx * 4 + j < live;
            const int col_rel = !bias || !on ? 0 : DKV ? rel_q(a, col) : -rel_k(a, col);
            const float col_lse = DKV && on ? __ldg(lse2 + col) : 0.0f;
            const float col_delta = DKV && on ? __ldg(delta + col) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float b = bias && on ? __ldg(bias + row_rel[i] + col_rel) : 0.0f;
                const float lse = DKV ? col_lse : row_lse[i], del = DKV ? col_delta : row_delta[i];
                const float w = on ? exp2_approx(fmaf(at(s, i, j), c2, b) - lse) : 0.0f;
                at(s, i, j) = w;
                at(d, i, j) = on ? w * (at(d, i, j) - del) : 0.0f;
            }
        }
        __syncthreads();
        if (DKV) simt_store_t(t1, s, ty, tx);
        simt_store_t(t2, d, ty, tx);
        __syncthreads();
        if (with_rel) {
            float ds[kRelHalf];
#pragma unroll
            for (int c = 0; c < kRelHalf; ++c)
                ds[c] = t2[(warp % 2 * kRelHalf + c) * kSimtPitch + warp / 2 * 32 + threadIdx.x % 32];
            const int col = min(j0 + warp % 2 * kRelHalf + (int)threadIdx.x % 32, keys - 1);
            const bool last = live <= kSimtTile;
            win.add(ds, live, rel_k(a, col), last ? 0 : rel_k(a, j0 + kSimtTile), last, rel_out);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c)
            if (c * 64 + tx * 4 < D) {
                const int K_ = min(live, kSimtTile);
                simt_product(acc1[c], t2 + ty * 4, kSimtPitch, n1 + c * 64 + tx * 4, pitch_n, K_);
                if (DKV)
                    simt_product(acc2[c], t1 + ty * 4, kSimtPitch, n2 + c * 64 + tx * 4, pitch_n, K_);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = i0 + ty * 4 + i;
        if (row >= rows) continue;
        const bool on = row < live_rows;   // rows of masked keys get zeros
        const int64_t at_row = (((int64_t)n * rows + row) * a.H + h) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = c * 64 + tx * 4 + j;
                if (d >= D) continue;
                ((T *)(DKV ? p.dK : p.dQ))[at_row + d] = IO<T>::st(on ? at(acc1[c], i, j) * a.scale : 0.0f);
                if (DKV) ((T *)p.dV)[at_row + d] = IO<T>::st(on ? at(acc2[c], i, j) : 0.0f);
            }
    }
}

// Whether every row of the operands starts at a multiple of 16 bytes.
template <typename T> bool simt_vec(const AttnArgs &a, const AttnPtrs &p) {
    constexpr int E = kVec<T>;
    bool vec = a.D % E == 0;
    for (const void *x : {p.Q, p.K, p.V, p.dO}) vec = vec && aligned16(x);
    for (int d = 0; d < 3; ++d)
        vec = vec && a.qs[d] % E == 0 && a.ks[d] % E == 0 && a.vs[d] % E == 0;
    return vec;
}

template <typename T>
cudaError_t launch_attn_simt_fwd(const AttnArgs &a, const AttnPtrs &p, const float *bias,
                                 cudaStream_t s) {
    const bool wide = a.D > 64, vec = simt_vec<T>(a, p);
    auto kernel = wide ? (vec ? attn_simt_fwd_kernel<T, 2, kVec<T>> : attn_simt_fwd_kernel<T, 2, 1>)
                       : (vec ? attn_simt_fwd_kernel<T, 1, kVec<T>> : attn_simt_fwd_kernel<T, 1, 1>);
    static DeviceFlags ready[2][2];
    const cudaError_t e = once_per_device(ready[wide][vec], [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    simt_fwd_smem(wide ? 128 : 64));
    });
    if (e != cudaSuccess) return e;
    const int64_t blocks = (int64_t)((a.Lq + kSimtTile - 1) / kSimtTile) * a.H * a.N;
    kernel<<<(unsigned)blocks, kSimtThreads, simt_fwd_smem(a.D), s>>>(a, p, bias);
    return cudaGetLastError();
}

// The key blocks, then the query blocks: one launch, so that either fills the
// SMs that the other leaves.
template <typename T, int NC, int E>
__global__ void __launch_bounds__(kSimtThreads)
    attn_simt_bwd_kernel(AttnArgs a, AttnPtrs p, const float *bias, const float *lse2,
                         const float *delta, RelArgs rel, int kv_blocks) {
    if ((int)blockIdx.x < kv_blocks)
        attn_simt_bwd_block<T, NC, E, true>(a, p, bias, lse2, delta, RelArgs(), blockIdx.x);
    else
        attn_simt_bwd_block<T, NC, E, false>(a, p, bias, lse2, delta, rel, blockIdx.x - kv_blocks);
}

// dK and dV of `kv_heads` (batch, head) pairs and dQ of `q_heads` from
// rel.head0 on (either may be 0).
template <typename T>
cudaError_t launch_attn_simt_bwd(const AttnArgs &a, const AttnPtrs &p, const float *bias,
                                 const float *lse2, const float *delta, const RelArgs &rel,
                                 int kv_heads, int q_heads, cudaStream_t s) {
    const bool wide = a.D > 64, vec = simt_vec<T>(a, p);
    auto kernel = wide ? (vec ? attn_simt_bwd_kernel<T, 2, kVec<T>> : attn_simt_bwd_kernel<T, 2, 1>)
                       : (vec ? attn_simt_bwd_kernel<T, 1, kVec<T>> : attn_simt_bwd_kernel<T, 1, 1>);
    static DeviceFlags ready[2][2];
    const cudaError_t e = once_per_device(ready[wide][vec], [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    227 * 1024 - 256);
    });
    if (e != cudaSuccess) return e;
    const int kv_blocks = (a.Lk + kSimtTile - 1) / kSimtTile * kv_heads;
    const int q_blocks = (a.Lq + kSimtTile - 1) / kSimtTile * q_heads;
    const int smem = std::max(simt_bwd_smem(a.D, true, 0), simt_bwd_smem(a.D, false, rel.window));
    kernel<<<(unsigned)kv_blocks + (unsigned)q_blocks, kSimtThreads, smem, s>>>(a, p, bias, lse2, delta,
                                                                               rel, kv_blocks);
    return cudaGetLastError();
}

}  // namespace gs
