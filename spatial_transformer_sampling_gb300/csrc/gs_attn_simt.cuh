// gs_attn_simt.cuh -- attention forward and backward in fp32 arithmetic, for
// fp32 tensors and for 16-bit ones whose rows the tensor-core kernels cannot
// take (head widths or strides that are not multiples of 16 bytes).
//
// 64 x 64 score tiles, four warps of 32 x 32, a thread 8 x 4 values, every
// product as a register-tiled outer product over operands in shared memory laid
// out contraction-major ([k][64 + 4]): per step three 16-byte shared loads feed
// sixteen packed FMAs.  A half-warp's lanes ask for 32 or 128 distinct bytes, one
// pass through shared memory each; with 4 x 4 values in rows of 16 lanes the
// loads took two thirds of its time and bound the kernels.  A tile's operands are
// fetched into registers in one batch, since with two or three blocks per SM
// the latency of loads in several batches showed.  Both together (4 images,
// 8 heads, 48 x 48 tokens, D 64, fp32): forward 1504 -> 1319 us, backward 4872 ->
// 4081 us; with the operands of a step read from shared memory one step ahead
// 1244 us (35 TFLOP/s of about 75 that the FMA units have) and 3906 us (28).  Rows
// (queries; keys in the dK / dV blocks) stay resident, columns are walked tile by
// tile; weights and their gradients go back through shared memory, over the
// columns' transposed copy, as the first operand of the next product.  One block
// sums each gradient in one order.
#pragma once

#include <cooperative_groups.h>

#include "gs_attn_common.cuh"
#include "gs_attn_rel.cuh"
#include "gs_ptx.cuh"
#include "gs_vec.cuh"

namespace gs {

constexpr int kSimtTile = 64;
constexpr int kSimtThreads = 128;
constexpr int kSimtMaxSplit = 8;   // blocks that share the keys of 64 queries (forward)
constexpr int kSimtPitch = kSimtTile + 4;   // keeps 16-byte alignment, spreads banks

// Element offsets of one operand: base + n, h, token strides.
template <typename T> struct SimtView {
    const T *p;
    int64_t by_token;
    __device__ __forceinline__ SimtView(const void *base, const int64_t (&s)[3], int n, int h)
        : p((const T *)base + n * s[0] + h * s[2]), by_token(s[1]) {}
};

// 64 tokens of an operand on their way from device memory: fetched into
// registers (by the backward kernel while the products of the tile before run),
// then put into shared memory token-major or contraction-major, or both.  A warp takes 16 tokens, two
// runs of V elements side by side: a 32-byte sector each, and no two lanes of a
// store in one bank.  Tokens from `live` on are zeros.
template <typename T, int NC, int V> struct SimtTokens {
    static constexpr int kRuns = 64 * NC / (2 * V);
    typename Run<T, V>::Raw r[kRuns];

    static __device__ __forceinline__ int token() {
        return threadIdx.x / 32 * 16 + threadIdx.x % 16;
    }
    static __device__ __forceinline__ int first(int k) { return (threadIdx.x / 16 % 2 + 2 * k) * V; }

    __device__ __forceinline__ void fetch(const SimtView<T> &v, int row0, int live, int D) {
        const T *p = v.p + (int64_t)(row0 + token()) * v.by_token;
        const bool on = token() < live;
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            r[k] = Run<T, V>::zero();
            if (on && first(k) < D) r[k] = Run<T, V>::load(p + first(k));
        }
    }
    // dst[d][64]
    __device__ __forceinline__ void put_t(float *dst, int D) const {
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            float x[V];
            Run<T, V>::widen(r[k], x);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (first(k) < D) dst[(first(k) + e) * kSimtPitch + token()] = x[e];
        }
    }
    // dst[64][pitch]
    __device__ __forceinline__ void put_n(float *dst, int pitch, int D) const {
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            float x[V];
            Run<T, V>::widen(r[k], x);
            float *at = dst + token() * pitch + first(k);
            if (first(k) >= D) continue;
            if constexpr (V == 1) {
                at[0] = x[0];
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 4)
                    *reinterpret_cast<float4 *>(at + e) =
                        make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            }
        }
    }
};

// A thread's place in the block's tile: eight rows from `row` on, four columns
// from `col` on.
struct SimtPlace {
    int row, col;
    __device__ __forceinline__ SimtPlace() {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        row = warp / 2 * 32 + lane / 8 * 8;
        col = warp % 2 * 32 + lane % 8 * 4;
    }
};

// c[8 rows][4] += sum_k a[k][8 rows] b[k][4 columns].  Pairs of rows share a
// packed FMA: the operand to be doubled is then the one of four values.  The next
// step's operands are read ahead, after the last one those of the row behind
// (kSimtBehind).
__device__ __forceinline__ void simt_product(float2 (&c)[4][4], const float *a, int pitch_a,
                                             const float *b, int pitch_b, int K) {
    float4 x = *reinterpret_cast<const float4 *>(a), z = *reinterpret_cast<const float4 *>(a + 4),
           y = *reinterpret_cast<const float4 *>(b);
#pragma unroll 8
    for (int k = 0; k < K; ++k) {
        const float2 r[4] = {make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(z.x, z.y),
                             make_float2(z.z, z.w)};
        const float w[4] = {y.x, y.y, y.z, y.w};
        a += pitch_a;
        b += pitch_b;
        x = *reinterpret_cast<const float4 *>(a);
        z = *reinterpret_cast<const float4 *>(a + 4);
        y = *reinterpret_cast<const float4 *>(b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                c[i][j] = fma_f32x2(r[i], make_float2(w[j], w[j]), c[i][j]);
    }
}

__device__ __forceinline__ float &at(float2 (&c)[4][4], int i, int j) {
    return i % 2 ? c[i / 2][j].y : c[i / 2][j].x;
}

// Stores the transpose of the block's 64 x 64 tile: dst[column][row].
__device__ __forceinline__ void simt_store_t(float *dst, float2 (&c)[4][4], const SimtPlace &me) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<float4 *>(dst + (me.col + j) * kSimtPitch + me.row + i) =
                make_float4(at(c, i, j), at(c, i + 1, j), at(c, i + 2, j), at(c, i + 3, j));
}

// Over the eight lanes that share a thread's rows.
__device__ __forceinline__ float row_lanes_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_lanes_sum(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Floats behind the last operand that are read but not used.
constexpr int kSimtBehind = 192;
static_assert(kSimtBehind >= kSimtPitch && kSimtBehind >= 128 + 8, "one row of either layout");

__host__ __device__ inline int simt_pitch_n(int D) { return (D + 3) / 4 * 4 + 4; }
// A transposed operand; one that weights are written over holds 64 rows at least.
__host__ __device__ inline int simt_floats_t(int D, bool reused) {
    return (reused && D < kSimtTile ? kSimtTile : D) * kSimtPitch;
}
inline int simt_fwd_smem(int D) {
    return (simt_floats_t(D, false) + simt_floats_t(D, true) + kSimtTile * simt_pitch_n(D) +
            kSimtBehind) * 4;
}
inline int simt_bwd_smem(int D, bool dkv, int rel) {
    return (2 * simt_floats_t(D, false) + 2 * simt_floats_t(D, true) +
            (dkv ? 2 : 1) * kSimtTile * simt_pitch_n(D) + kSimtBehind) * 4 + rel_smem(rel, 2);
}

// NC: 64-column chunks of the head width.  Three blocks per SM without fetching
// ahead beat two that do, 1319 to 1413 us at the size above.
template <typename T, int NC, int E, bool SPLIT>
__global__ void __launch_bounds__(kSimtThreads, NC == 1 ? 3 : 2)
    attn_simt_fwd_kernel(AttnArgs a, AttnPtrs p, const float *bias) {
    extern __shared__ float4 simt_smem[];
    const int D = a.D, pitch_n = simt_pitch_n(D);
    float *qt = reinterpret_cast<float *>(simt_smem), *kt = qt + simt_floats_t(D, false);
    float *vn = kt + simt_floats_t(D, true);
    const int tiles = (a.Lq + kSimtTile - 1) / kSimtTile;
    // SPLIT: a cluster shares the keys of 64 queries, whole tiles each
    const int splits = SPLIT ? cluster_size() : 1, block = blockIdx.x / splits;
    const int i0 = block % tiles * kSimtTile, h = block / tiles % a.H, n = block / tiles / a.H;
    const SimtPlace me;
    // of the columns' two halves, for a row's maximum and its sum
    __shared__ float s_half[2][kSimtTile];
    const int side = me.col / 32;
    const bool speaks = threadIdx.x % 8 == 0;   // for the eight lanes of its rows
    const float c2 = a.scale * kLog2e;
    const SimtView<T> Q(p.Q, a.qs, n, h), K(p.K, a.ks, n, h), V(p.V, a.vs, n, h);
    const int all_keys = keys_of(a, n);
    const int share = ((all_keys + kSimtTile - 1) / kSimtTile + splits - 1) / splits * kSimtTile;
    const int first = SPLIT ? cluster_rank() * share : 0;
    const int keys = SPLIT ? min(all_keys, first + share) : all_keys;
    wait_for_previous_kernel(bias);
    if (bias) bias += (int64_t)h * a.bias_stride;

    SimtTokens<T, NC, E> next_k, next_v;
    next_k.fetch(Q, i0, a.Lq - i0, D);
    next_k.put_t(qt, D);
    float2 o[NC][4][4] = {};
    float m[8], l[8];
    int rq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
        rq[i] = bias ? rel_q(a, min(i0 + me.row + i, a.Lq - 1)) : 0;
    }
    for (int j0 = first; j0 < keys; j0 += kSimtTile) {
        const int live = keys - j0;
        __syncthreads();
        next_k.fetch(K, j0, live, D);
        if (NC == 1) next_v.fetch(V, j0, live, D);
        next_k.put_t(kt, D);
        if (NC == 2) next_v.fetch(V, j0, live, D);
        next_v.put_n(vn, pitch_n, D);
        __syncthreads();
        float2 s[4][4] = {};
        simt_product(s, qt + me.row, kSimtPitch, kt + me.col, kSimtPitch, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool on = me.col + j < live;
            const int rk = bias && on ? rel_k(a, j0 + me.col + j) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float b = bias && on ? __ldg(bias + rq[i] - rk) : 0.0f;
                at(s, i, j) = on ? fmaf(at(s, i, j), c2, b) : -INFINITY;
            }
        }
        float top[8], keep[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top[i] = row_lanes_max(
                fmaxf(fmaxf(at(s, i, 0), at(s, i, 1)), fmaxf(at(s, i, 2), at(s, i, 3))));
            if (speaks) s_half[side][me.row + i] = top[i];
        }
        __syncthreads();   // and kt is read
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float next = fmaxf(m[i], fmaxf(top[i], s_half[side ^ 1][me.row + i]));
            const float ref = next == -INFINITY ? 0.0f : next;   // no key yet: weights 0
            keep[i] = exp2_approx(m[i] - ref);
            m[i] = next;
            l[i] *= keep[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                at(s, i, j) = exp2_approx(at(s, i, j) - ref);
                l[i] += at(s, i, j);
            }
        }
        simt_store_t(kt, s, me);
        __syncthreads();
#pragma unroll
        for (int c = 0; c < NC; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[c][i][j] = mul_f32x2(o[c][i][j], make_float2(keep[2 * i], keep[2 * i + 1]));
            if (c * 64 + me.col < D)
                simt_product(o[c], kt + me.row, kSimtPitch, vn + c * 64 + me.col, pitch_n,
                             min(live, kSimtTile));
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        l[i] = row_lanes_sum(l[i]);
        if (speaks) s_half[side][me.row + i] = l[i];
    }
    __syncthreads();
    if constexpr (SPLIT) {
        // the block's share: the output over V, the maximum and the sum over the halves
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[i] = s_half[0][me.row + i] + s_half[1][me.row + i];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c * 64 + me.col + j < D)
                        vn[(me.row + i) * pitch_n + c * 64 + me.col + j] = at(o[c], i, j);
        }
        __syncthreads();
        if (me.col == 0)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s_half[0][me.row + i] = m[i];
                s_half[1][me.row + i] = l[i];
            }
        // each block joins its part of the rows, the shares in order
        const auto cluster = cooperative_groups::this_cluster();
        cluster.sync();
        const int rows = kSimtTile / splits;
        for (int k = threadIdx.x; k < rows * D; k += kSimtThreads) {
            const int row = cluster_rank() * rows + k / D, d = k % D;
            if (i0 + row >= a.Lq) break;
            float top = -INFINITY, sum = 0.0f, v = 0.0f;
            for (int r = 0; r < splits; ++r)
                top = fmaxf(top, *cluster.map_shared_rank(&s_half[0][row], r));
            for (int r = 0; r < splits; ++r) {
                const float its = *cluster.map_shared_rank(&s_half[0][row], r);
                const float of = *cluster.map_shared_rank(&s_half[1][row], r);
                if (its == -INFINITY && of == 0.0f) continue;   // no key (a row of NaN has some)
                const float f = exp2_approx(its - top);
                sum = fmaf(of, f, sum);
                v = fmaf(*cluster.map_shared_rank(&vn[row * pitch_n + d], r), f, v);
            }
            const int64_t at_row = (int64_t)n * a.Lq + i0 + row;
            ((T *)p.O)[(at_row * a.H + h) * D + d] = IO<T>::st(sum != 0.0f ? v / sum : 0.0f);
            if (d == 0 && p.lse)
                p.lse[((int64_t)n * a.H + h) * a.Lq + i0 + row] = lse_of(top, sum);
        }
        cluster.sync();   // shared memory stays until the others have read it
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // both halves add in the same order
        const float sum = s_half[0][me.row + i] + s_half[1][me.row + i];
        const float f = sum != 0.0f ? 1.0f / sum : 0.0f;
        const int row = i0 + me.row + i;
        if (row >= a.Lq) continue;
        T *out = (T *)p.O + (((int64_t)n * a.Lq + row) * a.H + h) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c * 64 + me.col + j < D)
                    out[c * 64 + me.col + j] = IO<T>::st(at(o[c], i, j) * f);
        if (me.col == 0 && p.lse)
            p.lse[((int64_t)n * a.H + h) * a.Lq + row] = lse_of(m[i], sum);
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
    const SimtPlace me;
    const int warp = threadIdx.x / 32;
    const float c2 = a.scale * kLog2e;
    const int64_t dense[3] = {(int64_t)a.Lq * a.H * D, (int64_t)a.H * D, D};
    const SimtView<T> Q(p.Q, a.qs, n, h), K(p.K, a.ks, n, h), V(p.V, a.vs, n, h), G(p.dO, dense, n, h);
    const SimtView<T> &R1 = DKV ? K : Q, &R2 = DKV ? V : G, &C1 = DKV ? Q : K, &C2 = DKV ? G : V;
    const int keys = keys_of(a, n);
    const int live_rows = DKV ? keys : a.Lq;
    const int cols = i0 < live_rows ? (DKV ? a.Lq : keys) : 0;
    wait_for_previous_kernel(lse2, delta, bias);
    lse2 += (int64_t)nh * rows64(a.Lq);
    delta += (int64_t)nh * rows64(a.Lq);
    if (bias) bias += (int64_t)h * a.bias_stride;

    // One head-width chunk leaves the registers to fetch the next tile early.
    constexpr bool kAhead = NC == 1;
    SimtTokens<T, NC, E> next1, next2;
    next1.fetch(R1, i0, live_rows - i0, D);
    next2.fetch(R2, i0, live_rows - i0, D);
    next1.put_t(r1, D);
    next2.put_t(r2, D);
    if (kAhead) {
        next1.fetch(C1, 0, cols, D);
        next2.fetch(C2, 0, cols, D);
    }
    float2 acc1[NC][4][4] = {}, acc2[NC][4][4] = {};
    float row_lse[8], row_delta[8];
    int row_rel[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = min(i0 + me.row + i, max(live_rows - 1, 0));
        row_lse[i] = DKV ? 0.0f : lse2[row];
        row_delta[i] = DKV ? 0.0f : delta[row];
        row_rel[i] = !bias ? 0 : DKV ? -rel_k(a, row) : rel_q(a, row);
    }
    // two warps per 32 queries see to the bias gradient
    const bool with_rel = !DKV && rel.window > 0 && i0 + warp / 2 * 32 < a.Lq && cols > 0;
    RelWindow win;
    float *rel_out = nullptr;
    if (with_rel) rel_out = win.init(a, win_smem, rel, i0, nh, warp / 2, warp % 2);

    for (int j0 = 0; j0 < cols; j0 += kSimtTile) {
        const int live = cols - j0;
        __syncthreads();
        if (!kAhead) next1.fetch(C1, j0, live, D);
        next1.put_t(t1, D);
        next1.put_n(n1, pitch_n, D);
        if (!kAhead) next2.fetch(C2, j0, live, D);
        next2.put_t(t2, D);
        if (DKV) next2.put_n(n2, pitch_n, D);
        __syncthreads();
        float2 s[4][4] = {}, d[4][4] = {};
        simt_product(s, r1 + me.row, kSimtPitch, t1 + me.col, kSimtPitch, D);
        simt_product(d, r2 + me.row, kSimtPitch, t2 + me.col, kSimtPitch, D);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = j0 + me.col + j;
            const bool on = me.col + j < live;
            const int col_rel = !bias || !on ? 0 : DKV ? rel_q(a, col) : -rel_k(a, col);
            const float col_lse = DKV && on ? __ldg(lse2 + col) : 0.0f;
            const float col_delta = DKV && on ? __ldg(delta + col) : 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float b = bias && on ? __ldg(bias + row_rel[i] + col_rel) : 0.0f;
                const float lse = DKV ? col_lse : row_lse[i], del = DKV ? col_delta : row_delta[i];
                const float w = on ? exp2_approx(fmaf(at(s, i, j), c2, b) - lse) : 0.0f;
                at(s, i, j) = w;
                at(d, i, j) = on ? w * (at(d, i, j) - del) : 0.0f;
            }
        }
        __syncthreads();
        if (DKV) simt_store_t(t1, s, me);
        simt_store_t(t2, d, me);
        __syncthreads();
        if (kAhead) {
            next1.fetch(C1, j0 + kSimtTile, live - kSimtTile, D);
            next2.fetch(C2, j0 + kSimtTile, live - kSimtTile, D);
        }
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
            if (c * 64 + me.col < D) {
                const int K_ = min(live, kSimtTile);
                simt_product(acc1[c], t2 + me.row, kSimtPitch, n1 + c * 64 + me.col, pitch_n, K_);
                if (DKV)
                    simt_product(acc2[c], t1 + me.row, kSimtPitch, n2 + c * 64 + me.col, pitch_n, K_);
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i0 + me.row + i;
        if (row >= rows) continue;
        const bool on = row < live_rows;   // rows of masked keys get zeros
        const int64_t at_row = (((int64_t)n * rows + row) * a.H + h) * D;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = c * 64 + me.col + j;
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
    constexpr int E = kVec<T>;
    const bool wide = a.D > 64, vec = simt_vec<T>(a, p);
    // Few blocks of long heads: several for one, of two key tiles at least, up to a
    // quarter more blocks than SMs (3000 tokens, one head, D 64, fp32: 107 us, 209
    // with one each; 17 x 23 tokens, 4 x 4 heads, from 112 blocks to 224: 41 to 51).
    const int64_t blocks = (int64_t)((a.Lq + kSimtTile - 1) / kSimtTile) * a.H * a.N;
    const int tiles = (a.Lk + kSimtTile - 1) / kSimtTile;
    int splits = 1;
    while (splits < kSimtMaxSplit && blocks * splits * 2 <= 152 + 152 / 4 && tiles >= splits * 4)
        splits *= 2;
    const bool split = splits > 1;
    auto kernel =
        split ? (wide ? (vec ? attn_simt_fwd_kernel<T, 2, E, true> : attn_simt_fwd_kernel<T, 2, 1, true>)
                      : (vec ? attn_simt_fwd_kernel<T, 1, E, true> : attn_simt_fwd_kernel<T, 1, 1, true>))
              : (wide ? (vec ? attn_simt_fwd_kernel<T, 2, E, false> : attn_simt_fwd_kernel<T, 2, 1, false>)
                      : (vec ? attn_simt_fwd_kernel<T, 1, E, false> : attn_simt_fwd_kernel<T, 1, 1, false>));
    static DeviceFlags ready[2][2][2];
    const cudaError_t e = once_per_device(ready[split][wide][vec], [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    simt_fwd_smem(wide ? 128 : 64));
    });
    if (e != cudaSuccess) return e;
    return launch_next(LaunchAs(bias != nullptr, splits), kernel, (unsigned)(blocks * splits),
                       kSimtThreads, simt_fwd_smem(a.D), s, a, p, bias);
}

// The key blocks, then the query blocks: one launch, so that either fills the
// SMs that the other leaves, the longer ones (four products of 64 x 64 x D a step,
// not three) first.
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
    return launch_next(true, kernel, (unsigned)kv_blocks + (unsigned)q_blocks, kSimtThreads, smem, s, a,
                       p, bias, lse2, delta, rel, kv_blocks);
}

}  // namespace gs
