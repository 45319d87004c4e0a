// gs_attn.cuh -- attention with a learned bias by relative position: which
// kernel takes a call, and the steps around them.
//
//   s[n,h,i,j] = scale * q[n,i,h] . k[n,j,h] + table[bucket(i, j)][h]
//   p = softmax over j,  o = sum_j p v,  lse = log sum_j exp(s)
// Backward, with delta_i = do_i . o_i:
//   ds = p * (do_i . v_j - delta_i),  dq_i = scale sum_j ds k_j,
//   dk_j = scale sum_i ds q_i,  dv_j = sum_i p do_i,
//   dtable[b][h] = sum of ds over the batch and the pairs of bucket b.
//
// Forward: up to kFewQueries queries run on attn_few_kernel, which reads K and
// V once and splits the keys over a cluster.  Otherwise 16-bit types whose rows
// TMA can read run on the tensor cores, the rest on fp32 FMAs.  The bias is
// expanded once per call to (H, R) in base-2 units, R relative indices, so that
// the kernels look up one float per pair.
#pragma once

#include "gs_attn_common.cuh"
#include "gs_attn_few.cuh"
#include "gs_attn_simt.cuh"
#include "gs_attn_tc_bwd.cuh"
#include "gs_attn_tc_fwd.cuh"

namespace gs {
namespace {

// bias[h][pad + r] for every relative index, in base-2 units, and zeros around: 2 us
// for 3969 indices and 8 heads, the latency of a bucket and its entry.
template <typename T>
__global__ void attn_bias_kernel(const T *table, AttnArgs a, int pad, float *bias) {
    const int at = blockIdx.x * blockDim.x + threadIdx.x, r = at - pad;
    if (at >= a.bias_stride) return;
    const int b = r >= 0 && r < a.R ? __ldg(a.buckets + r) : 0;
    for (int h = blockIdx.y; h < a.H; h += gridDim.y)
        bias[(int64_t)h * a.bias_stride + at] =
            r >= 0 && r < a.R ? bias2_of(table, b, a.nb, a.H, h) : 0.0f;
}

// Sum of ds over the batch and the pairs of one relative index, one warp per
// index: for the grids whose indices do not fit the query kernels' windows.
template <typename T>
__global__ void attn_dbias_kernel(AttnArgs a, AttnPtrs p, const float *bias, const float *lse2,
                                  const float *delta, float *rel) {
    wait_for_previous_kernel(bias, lse2, delta);
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
    const int lane = threadIdx.x % 32;
    if (w >= (int64_t)a.H * a.R) return;
    const int r = (int)(w % a.R), h = (int)(w / a.R);
    const int dy = r / a.P - (a.Hk - 1), dx = r % a.P - (a.Wk - 1);
    const float b = __ldg(bias + (int64_t)h * a.bias_stride + r);
    float sum = 0.0f;
    for (int n = 0; n < a.N && b != -INFINITY; ++n) {
        const int keys = keys_of(a, n);
        const T *q = (const T *)p.Q + n * a.qs[0] + h * a.qs[2];
        const T *k = (const T *)p.K + n * a.ks[0] + h * a.ks[2];
        const T *v = (const T *)p.V + n * a.vs[0] + h * a.vs[2];
        const T *g = (const T *)p.dO + ((int64_t)n * a.Lq * a.H + h) * a.D;
        const int64_t row0 = ((int64_t)n * a.H + h) * rows64(a.Lq);
        for (int y = max(0, dy); y < min(a.Hq, a.Hk + dy); ++y)
            for (int x = max(0, dx); x < min(a.Wq, a.Wk + dx); ++x) {
                const int i = y * a.Wq + x, j = (y - dy) * a.Wk + x - dx;
                if (j >= keys) continue;
                float s = 0.0f, dp = 0.0f;
                for (int d = lane; d < a.D; d += 32) {
                    s = fmaf(IO<T>::ld(q + i * a.qs[1] + d), IO<T>::ld(k + j * a.ks[1] + d), s);
                    dp = fmaf(IO<T>::ld(g + (int64_t)i * a.H * a.D + d),
                              IO<T>::ld(v + j * a.vs[1] + d), dp);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                    dp += __shfl_xor_sync(0xffffffffu, dp, o);
                }
                sum += exp2_approx(fmaf(s, a.scale * kLog2e, b) - lse2[row0 + i]) *
                       (dp - delta[row0 + i]);
            }
    }
    if (lane == 0) rel[w] = sum;
}

// dtable[b][h]: a lane per bucket goes through the relative indices in order,
// sixteen warps a share each of what shared memory holds at a time.  4.7 us for
// 3969 indices, 256 buckets, 8 heads (eight warps: 6.6): two passes' latency.
constexpr int kTableThreads = 512;
template <typename T>
__global__ void __launch_bounds__(kTableThreads) attn_dtable_kernel(AttnArgs a, const float *rel, T *dTable) {
    constexpr int kWarps = kTableThreads / 32, kHeld = 4096, kShare = kHeld / kWarps;
    __shared__ __align__(16) int2 s_pair[kHeld];   // bucket, bits of the sum
    __shared__ float s_sum[kWarps][32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, h = blockIdx.y;
    const int b = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    wait_for_previous_kernel(rel);
    for (int r0 = 0; r0 < a.R; r0 += kHeld) {
        __syncthreads();
        for (int k = threadIdx.x; k < kHeld; k += kTableThreads)
            s_pair[k] = r0 + k < a.R ? make_int2(__ldg(a.buckets + r0 + k),
                                                 __float_as_int(rel[(int64_t)h * a.R + r0 + k]))
                                     : make_int2(-1, 0);
        __syncthreads();
        const int4 *at = reinterpret_cast<const int4 *>(s_pair + warp * kShare);
        const int count = min(max(a.R - r0 - warp * kShare, 0), kShare);
#pragma unroll 8
        for (int k = 0; k < (count + 1) / 2; ++k) {
            const int4 v = at[k];
            if (v.x == b) sum += __int_as_float(v.y);
            if (v.z == b) sum += __int_as_float(v.w);
        }
    }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && b < a.nb) {
        for (int w = 1; w < kWarps; ++w) sum += s_sum[w][lane];
        dTable[(int64_t)b * a.H + h] = IO<T>::st(sum);
    }
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Floats per head of the expanded bias.
int bias_stride(const AttnArgs &a) { return (a.R + 3) / 4 * 4 + 2 * tc_bias_pad(a); }

// The workspace's parts, in order; offsets in bytes.
struct Workspace {
    size_t bias, rel, lse2, delta, range, part, end;
};
template <typename T> Workspace workspace_of(const AttnArgs &a, bool backward) {
    Workspace w = {};
    if (!backward && few_takes(a)) return w;
    const size_t per_rel = a.nb ? round256((size_t)a.H * a.R * sizeof(float)) : 0;
    w.rel = w.end = a.nb ? round256((size_t)a.H * bias_stride(a) * sizeof(float)) : 0;
    if (!backward) return w;
    const size_t per_row = round256((size_t)a.N * a.H * rows64(a.Lq) * sizeof(float));
    w.lse2 = w.rel + per_rel;
    w.delta = w.lse2 + per_row;
    w.range = w.delta + per_row;
    w.part = w.end = w.range + (kScaledGradient<T> ? round256((size_t)a.N * a.H * range_parts(a) * 2 *
                                                              sizeof(float))
                                                   : 0);
    if (a.nb && rel_window_of(a) > 0)
        w.end += round256((size_t)rel_heads_of(a) * ((a.Lq + 31) / 32) * rel_stride_of(a) *
                          sizeof(float));
    return w;
}

// Fills the expanded bias; *entry_0: the entry of relative index 0 of head 0.
template <typename T>
cudaError_t expand_bias(AttnArgs &a, const AttnPtrs &p, char *ws, const float **entry_0, cudaStream_t s) {
    *entry_0 = nullptr;
    if (a.nb == 0) return cudaSuccess;
    float *bias = (float *)(ws + workspace_of<T>(a, false).bias);
    const int pad = tc_bias_pad(a);
    a.bias_stride = bias_stride(a);
    *entry_0 = bias + pad;
    return launch_next(false, attn_bias_kernel<T>, dim3((a.bias_stride + 255) / 256, a.H), 256, 0, s,
                       (const T *)p.table, a, pad, bias);
}

// Tensor-core views of the backward pass (16-bit types); false when its kernels
// do not take the call (rows that are not multiples of 16 bytes).
template <typename T>
bool tc_backward_views(const AttnArgs &a, const AttnPtrs &ptr, TcBwdArgs &kv, TcBwdArgs &q) {
    if (a.D % 8 != 0) return false;
    for (const void *p : {(const void *)ptr.O, ptr.dO, (const void *)ptr.dQ, (const void *)ptr.dK,
                          (const void *)ptr.dV})
        if ((uintptr_t)p & 15u) return false;
    constexpr bool bf16 = __is_same(T, __nv_bfloat16);
    const int64_t dense[3] = {(int64_t)a.Lq * a.H * a.D, (int64_t)a.H * a.D, a.D};
    return tc_view(&kv.r1, ptr.K, bf16, a.N, a.Lk, a.H, a.D, a.ks, kTcM) &&
           tc_view(&kv.r2, ptr.V, bf16, a.N, a.Lk, a.H, a.D, a.vs, kTcM) &&
           tc_view(&kv.c1, ptr.Q, bf16, a.N, a.Lq, a.H, a.D, a.qs, kTcN) &&
           tc_view(&kv.c2, ptr.dO, bf16, a.N, a.Lq, a.H, a.D, dense, kTcN) &&
           tc_view(&q.r1, ptr.Q, bf16, a.N, a.Lq, a.H, a.D, a.qs, kTcM) &&
           tc_view(&q.r2, ptr.dO, bf16, a.N, a.Lq, a.H, a.D, dense, kTcM) &&
           tc_view(&q.c1, ptr.K, bf16, a.N, a.Lk, a.H, a.D, a.ks, kTcN) &&
           tc_view(&q.c2, ptr.V, bf16, a.N, a.Lk, a.H, a.D, a.vs, kTcN);
}

}  // namespace

template <typename T>
size_t attn_ws_bytes(const AttnArgs &a, bool backward) {
    return workspace_of<T>(a, backward).end;
}

template <typename T>
cudaError_t launch_attn(const AttnArgs &args, const AttnPtrs &p, void *ws, cudaStream_t s) {
    AttnArgs a = args;
    if (few_takes(a)) return launch_attn_few<T>(a, p, s);
    const float *bias;
    cudaError_t e = expand_bias<T>(a, p, (char *)ws, &bias, s);
    if (e != cudaSuccess) return e;
    if constexpr (sizeof(T) == 2) {
        bool used = false;
        e = launch_attn_tc_fwd<T>(a, p, bias, s, &used);
        if (used || e != cudaSuccess) return e;
    }
    return launch_attn_simt_fwd<T>(a, p, bias, s);
}

template <typename T>
cudaError_t launch_attn_backward(const AttnArgs &args, const AttnPtrs &p, void *ws_, cudaStream_t s) {
    AttnArgs a = args;
    char *ws = (char *)ws_;
    const Workspace w = workspace_of<T>(a, true);
    const float *bias;
    cudaError_t e = expand_bias<T>(a, p, ws, &bias, s);
    if (e != cudaSuccess) return e;
    float *rel = (float *)(ws + w.rel), *lse2 = (float *)(ws + w.lse2);
    float *delta = (float *)(ws + w.delta);
    TcBwdArgs kv, q;
    bool tc = false;
    if constexpr (sizeof(T) == 2) tc = tc_backward_views<T>(a, p, kv, q);
    const int pairs = a.N * a.H;
    RangeArgs range = {};
    if (kScaledGradient<T> && tc) range = {range_parts(a), (float *)(ws + w.range)};
    e = launch_attn_delta<T>(a, p, lse2, delta, range, s);
    if (e != cudaSuccess) return e;
    RelArgs part = {};
    part.window = bias ? rel_window_of(a) : 0;
    part.stride = part.window ? (int)rel_stride_of(a) : 0;
    part.part = (float *)(ws + w.part);
    if (tc) {
        kv.a = q.a = a;
        kv.bias = tc_bias_of(a, true);
        q.bias = tc_bias_of(a, false);
        kv.bias.base = q.bias.base = bias;
        kv.bias.stride = q.bias.stride = a.bias_stride;
        kv.lse2 = q.lse2 = lse2;
        kv.delta = q.delta = delta;
        kv.range = q.range = range;
        kv.out1 = p.dK;
        kv.out2 = p.dV;
        q.out1 = p.dQ;
        q.out2 = nullptr;
        kv.rel = RelArgs();
    }
    const int heads = part.window ? (int)rel_heads_of(a) : pairs;
    for (part.head0 = 0; part.head0 < pairs; part.head0 += heads) {
        const int now = std::min(heads, pairs - part.head0);
        const int kv_heads = part.head0 == 0 ? pairs : 0;
        q.rel = part;
        e = cudaErrorInvalidValue;
        if constexpr (sizeof(T) == 2)
            if (tc) e = launch_attn_tc_bwd<T>(kv, q, kv_heads, now, s);
        if (!tc) e = launch_attn_simt_bwd<T>(a, p, bias, lse2, delta, part, kv_heads, now, s);
        if (e != cudaSuccess) return e;
        if (part.window)
            e = launch_next(true, attn_rel_sum_kernel, dim3((a.R + kRelSumIndices - 1) / kRelSumIndices, a.H),
                            kRelSumThreads, 0, s, a, part, now, rel);
        if (e != cudaSuccess) return e;
    }
    if (bias) {
        if (!part.window)
            e = launch_next(true, attn_dbias_kernel<T>, (unsigned)(((int64_t)a.H * a.R + 7) / 8), 256, 0, s,
                            a, p, bias, lse2, delta, rel);
        if (e != cudaSuccess) return e;
        e = launch_next(true, attn_dtable_kernel<T>, dim3((a.nb + 31) / 32, a.H), kTableThreads, 0, s, a,
                        rel, (T *)p.dTable);
    }
    return e;
}

}  // namespace gs
