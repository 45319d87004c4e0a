// gs_attn.cu -- attention with a learned bias by relative position, forward
// and backward: one warp per query, per key or per relative index.
//
//   s[n,h,i,j] = scale * q[n,i,h] . k[n,j,h] + table[bucket(i, j)][h]
//   p = softmax over j,  o = sum_j p v,  lse = log sum_j exp(s)
// Backward, with D_i = do_i . o_i:
//   ds = p * (do_i . v_j - D_i),  dq_i = scale sum_j ds k_j,
//   dk_j = scale sum_i ds q_i,  dv_j = sum_i p do_i,
//   dtable[b][h] = sum of ds over the batch and the pairs of bucket b.
#include "gs_attn_common.cuh"
#include "gs_attn_tc_bwd.cuh"
#include "gs_attn_tc_fwd.cuh"

namespace gs {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxDimsPerLane = 4;   // head widths to 128

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// bias[h][r] for every relative index, in base-2 units.
template <typename T>
__global__ void attn_bias_kernel(const T *table, AttnArgs a, float *bias) {
    const int r = blockIdx.x * blockDim.x + threadIdx.x;
    if (r >= a.R) return;
    const int b = __ldg(a.buckets + r);
    for (int h = blockIdx.y; h < a.H; h += gridDim.y)
        bias[(int64_t)h * a.R + r] = bias2_of(table, b, a.nb, a.H, h);
}

// This lane's slice of a row of D elements: dims lane, lane + 32, ...
template <typename T>
__device__ __forceinline__ void load_row(const T *p, int D, float (&v)[kMaxDimsPerLane]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int k = 0; k < kMaxDimsPerLane; ++k)
        v[k] = lane + 32 * k < D ? IO<T>::ld(p + lane + 32 * k) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_row(T *p, int D, const float (&v)[kMaxDimsPerLane], float f) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int k = 0; k < kMaxDimsPerLane; ++k)
        if (lane + 32 * k < D) p[lane + 32 * k] = IO<T>::st(v[k] * f);
}
__device__ __forceinline__ float dot(const float (&a)[kMaxDimsPerLane],
                                     const float (&b)[kMaxDimsPerLane]) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxDimsPerLane; ++k) s = fmaf(a[k], b[k], s);
    return warp_sum(s);
}
__device__ __forceinline__ void axpy(float f, const float (&x)[kMaxDimsPerLane],
                                     float (&y)[kMaxDimsPerLane]) {
#pragma unroll
    for (int k = 0; k < kMaxDimsPerLane; ++k) y[k] = fmaf(f, x[k], y[k]);
}

// Offset of a token's head row in a dense (N, L, H, D) tensor.
__device__ __forceinline__ int64_t dense_row(const AttnArgs &a, int L, int n, int i, int h) {
    return (((int64_t)n * L + i) * a.H + h) * a.D;
}

template <typename T>
__global__ void attn_fwd_kernel(AttnArgs a, AttnPtrs p, const float *bias) {
    const int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (w >= (int64_t)a.N * a.H * a.Lq) return;
    const int i = (int)(w % a.Lq), h = (int)(w / a.Lq % a.H), n = (int)(w / a.Lq / a.H);
    float q[kMaxDimsPerLane], o[kMaxDimsPerLane] = {};
    load_row((const T *)p.Q + n * a.qs[0] + i * a.qs[1] + h * a.qs[2], a.D, q);
    const int keys = keys_of(a, n), ri = rel_q(a, i);
    float m = -INFINITY, l = 0.0f;
    for (int j = 0; j < keys; ++j) {
        float k[kMaxDimsPerLane], v[kMaxDimsPerLane];
        const float b = bias ? __ldg(bias + (int64_t)h * a.R + ri - rel_k(a, j)) : 0.0f;
        if (b == -INFINITY) continue;
        load_row((const T *)p.K + n * a.ks[0] + j * a.ks[1] + h * a.ks[2], a.D, k);
        load_row((const T *)p.V + n * a.vs[0] + j * a.vs[1] + h * a.vs[2], a.D, v);
        const float s = fmaf(dot(q, k), a.scale * kLog2e, b);
        const float top = fmaxf(m, s);
        if (top == -INFINITY && s == -INFINITY) continue;   // a NaN score goes on
        const float keep = exp2_approx(m - top), e = exp2_approx(s - top);
        l = fmaf(l, keep, e);
#pragma unroll
        for (int d = 0; d < kMaxDimsPerLane; ++d) o[d] = fmaf(o[d], keep, e * v[d]);
        m = top;
    }
    store_row((T *)p.O + dense_row(a, a.Lq, n, i, h), a.D, o, l != 0.0f ? 1.0f / l : 0.0f);
    if (p.lse && threadIdx.x % 32 == 0)
        p.lse[((int64_t)n * a.H + h) * a.Lq + i] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

// p and ds of one pair, from the query's and the key's rows.
template <typename T>
struct Pair {
    float q[kMaxDimsPerLane], k[kMaxDimsPerLane], v[kMaxDimsPerLane], g[kMaxDimsPerLane];
    float lse2, delta;
    __device__ __forceinline__ void query(const AttnArgs &a, const AttnPtrs &p, int n, int h, int i) {
        const int64_t at = dense_row(a, a.Lq, n, i, h);
        float o[kMaxDimsPerLane];
        load_row((const T *)p.Q + n * a.qs[0] + i * a.qs[1] + h * a.qs[2], a.D, q);
        load_row((const T *)p.dO + at, a.D, g);
        load_row((const T *)p.O + at, a.D, o);
        lse2 = p.lse[((int64_t)n * a.H + h) * a.Lq + i] * kLog2e;
        delta = dot(g, o);
    }
    __device__ __forceinline__ void key(const AttnArgs &a, const AttnPtrs &p, int n, int h, int j) {
        load_row((const T *)p.K + n * a.ks[0] + j * a.ks[1] + h * a.ks[2], a.D, k);
        load_row((const T *)p.V + n * a.vs[0] + j * a.vs[1] + h * a.vs[2], a.D, v);
    }
    // p and ds; both 0 where the pair is masked or the row has no key at all
    __device__ __forceinline__ void weights(const AttnArgs &a, float b, float &pw, float &ds) const {
        const float s = fmaf(dot(q, k), a.scale * kLog2e, b);
        const float dp = dot(g, v);
        const bool live = b != -INFINITY && lse2 != -INFINITY;
        pw = live ? exp2_approx(s - lse2) : 0.0f;
        ds = live ? pw * (dp - delta) : 0.0f;
    }
};

template <typename T>
__global__ void attn_dq_kernel(AttnArgs a, AttnPtrs p, const float *bias) {
    const int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (w >= (int64_t)a.N * a.H * a.Lq) return;
    const int i = (int)(w % a.Lq), h = (int)(w / a.Lq % a.H), n = (int)(w / a.Lq / a.H);
    Pair<T> t;
    t.query(a, p, n, h, i);
    float dq[kMaxDimsPerLane] = {};
    const int keys = keys_of(a, n), ri = rel_q(a, i);
    for (int j = 0; j < keys; ++j) {
        const float b = bias ? __ldg(bias + (int64_t)h * a.R + ri - rel_k(a, j)) : 0.0f;
        if (b == -INFINITY) continue;
        float pw, ds;
        t.key(a, p, n, h, j);
        t.weights(a, b, pw, ds);
        axpy(ds, t.k, dq);
    }
    store_row((T *)p.dQ + dense_row(a, a.Lq, n, i, h), a.D, dq, a.scale);
}

template <typename T>
__global__ void attn_dkv_kernel(AttnArgs a, AttnPtrs p, const float *bias) {
    const int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (w >= (int64_t)a.N * a.H * a.Lk) return;
    const int j = (int)(w % a.Lk), h = (int)(w / a.Lk % a.H), n = (int)(w / a.Lk / a.H);
    Pair<T> t;
    float dk[kMaxDimsPerLane] = {}, dv[kMaxDimsPerLane] = {};
    if (j < keys_of(a, n)) {
        t.key(a, p, n, h, j);
        const int rj = rel_k(a, j);
        for (int i = 0; i < a.Lq; ++i) {
            const float b = bias ? __ldg(bias + (int64_t)h * a.R + rel_q(a, i) - rj) : 0.0f;
            if (b == -INFINITY) continue;
            float pw, ds;
            t.query(a, p, n, h, i);
            t.weights(a, b, pw, ds);
            axpy(ds, t.q, dk);
            axpy(pw, t.g, dv);
        }
    }
    const int64_t at = dense_row(a, a.Lk, n, j, h);
    store_row((T *)p.dK + at, a.D, dk, a.scale);
    store_row((T *)p.dV + at, a.D, dv, 1.0f);
}

// Sum of ds over the batch and the pairs of one relative index.
template <typename T>
__global__ void attn_dbias_kernel(AttnArgs a, AttnPtrs p, const float *bias, float *rel) {
    const int64_t w = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    if (w >= (int64_t)a.H * a.R) return;
    const int r = (int)(w % a.R), h = (int)(w / a.R);
    const int dy = r / a.P - (a.Hk - 1), dx = r % a.P - (a.Wk - 1);
    const float b = __ldg(bias + w);
    float sum = 0.0f;
    if (b != -INFINITY) {
        Pair<T> t;
        for (int n = 0; n < a.N; ++n) {
            const int keys = keys_of(a, n);
            for (int y = max(0, dy); y < min(a.Hq, a.Hk + dy); ++y)
                for (int x = max(0, dx); x < min(a.Wq, a.Wk + dx); ++x) {
                    const int i = y * a.Wq + x, j = (y - dy) * a.Wk + x - dx;
                    if (j >= keys) continue;
                    float pw, ds;
                    t.query(a, p, n, h, i);
                    t.key(a, p, n, h, j);
                    t.weights(a, b, pw, ds);
                    sum += ds;
                }
        }
    }
    if (threadIdx.x % 32 == 0) rel[w] = sum;
}

// dtable[b][h]: the relative indices of bucket b, in order.
template <typename T>
__global__ void attn_dtable_kernel(AttnArgs a, const float *rel, T *dTable) {
    const int w = blockIdx.x * kWarps + threadIdx.x / 32, lane = threadIdx.x % 32;
    if (w >= a.nb * a.H) return;
    const int h = w % a.H, b = w / a.H;
    float sum = 0.0f;
    for (int r = lane; r < a.R; r += 32)
        if (__ldg(a.buckets + r) == b) sum += rel[(int64_t)h * a.R + r];
    sum = warp_sum(sum);
    if (lane == 0) dTable[w] = IO<T>::st(sum);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
unsigned warp_blocks(int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); }

template <typename T>
const float *expand_bias(const AttnArgs &a, const AttnPtrs &p, void *ws, cudaStream_t s) {
    if (a.nb == 0) return nullptr;
    attn_bias_kernel<T><<<dim3((a.R + 255) / 256, a.H < 65535 ? a.H : 65535), 256, 0, s>>>(
        (const T *)p.table, a, (float *)ws);
    return (const float *)ws;
}

// The tensor-core kernels take 16-bit types and head widths that are multiples
// of 8 (their 16-byte rows); they also want aligned pointers and strides, which
// tc_view checks.
template <typename T> bool tc_takes(const AttnArgs &a) { return sizeof(T) == 2 && a.D % 8 == 0; }

// The workspace's parts, in order; offsets in bytes.
struct Workspace {
    size_t bias, rel, lse2, delta, part, end;
};
template <typename T> Workspace workspace_of(const AttnArgs &a, bool backward) {
    Workspace w;
    const size_t per_rel = a.nb ? round256((size_t)a.H * a.R * sizeof(float)) : 0;
    w.bias = 0;
    w.rel = w.bias + per_rel;
    w.lse2 = w.delta = w.part = w.end = w.rel;
    if (!backward) return w;
    w.lse2 = w.rel + per_rel;
    const bool tc = tc_takes<T>(a);
    const size_t per_row = tc ? round256((size_t)a.N * a.H * rows64(a.Lq) * sizeof(float)) : 0;
    w.delta = w.lse2 + per_row;
    w.part = w.delta + per_row;
    const bool rel = tc && a.nb && tc_rel_window(a) > 0;
    w.end = w.part + (rel ? round256((size_t)tc_rel_heads(a) * ((a.Lq + 31) / 32) *
                                     tc_rel_stride(a) * sizeof(float))
                          : 0);
    return w;
}

}  // namespace

template <typename T>
size_t attn_ws_bytes(const AttnArgs &a, bool backward) {
    return workspace_of<T>(a, backward).end;
}

namespace {

// The tensor-core backward pass; *used reports whether it takes the call, and
// *rel_done whether rel holds the bias gradient by relative index.
template <typename T>
cudaError_t launch_tc_backward(const AttnArgs &a, const AttnPtrs &ptr, const float *bias, char *ws,
                               cudaStream_t s, bool *used, bool *rel_done) {
    *used = *rel_done = false;
    if (!tc_takes<T>(a)) return cudaSuccess;
    for (const void *p : {(const void *)ptr.O, ptr.dO, (const void *)ptr.dQ, (const void *)ptr.dK,
                          (const void *)ptr.dV})
        if ((uintptr_t)p & 15u) return cudaSuccess;
    constexpr bool bf16 = __is_same(T, __nv_bfloat16);
    const int64_t dense[3] = {(int64_t)a.Lq * a.H * a.D, (int64_t)a.H * a.D, a.D};
    TcBwdArgs kv, q;   // keys against queries; queries against keys
    if (!tc_view(&kv.r1, ptr.K, bf16, a.N, a.Lk, a.H, a.D, a.ks, kTcM) ||
        !tc_view(&kv.r2, ptr.V, bf16, a.N, a.Lk, a.H, a.D, a.vs, kTcM) ||
        !tc_view(&kv.c1, ptr.Q, bf16, a.N, a.Lq, a.H, a.D, a.qs, kTcN) ||
        !tc_view(&kv.c2, ptr.dO, bf16, a.N, a.Lq, a.H, a.D, dense, kTcN) ||
        !tc_view(&q.r1, ptr.Q, bf16, a.N, a.Lq, a.H, a.D, a.qs, kTcM) ||
        !tc_view(&q.r2, ptr.dO, bf16, a.N, a.Lq, a.H, a.D, dense, kTcM) ||
        !tc_view(&q.c1, ptr.K, bf16, a.N, a.Lk, a.H, a.D, a.ks, kTcN) ||
        !tc_view(&q.c2, ptr.V, bf16, a.N, a.Lk, a.H, a.D, a.vs, kTcN))
        return cudaSuccess;
    *used = true;
    const Workspace w = workspace_of<T>(a, true);
    float *lse2 = (float *)(ws + w.lse2), *delta = (float *)(ws + w.delta);
    const int64_t rows = (int64_t)a.N * rows64(a.Lq) * a.H;
    attn_delta_kernel<T><<<(unsigned)((rows + 15) / 16), 256, 0, s>>>(
        a, (const T *)ptr.dO, (const T *)ptr.O, ptr.lse, lse2, delta);
    kv.a = q.a = a;
    kv.bias = q.bias = bias;
    kv.lse2 = q.lse2 = lse2;
    kv.delta = q.delta = delta;
    kv.out1 = ptr.dK;
    kv.out2 = ptr.dV;
    q.out1 = ptr.dQ;
    q.out2 = nullptr;
    kv.rel_window = kv.rel_stride = kv.head0 = 0;
    kv.rel_part = nullptr;
    const int pairs = a.N * a.H;
    cudaError_t e = launch_attn_tc_bwd_kernel<T, true>(kv, pairs, s);
    if (e != cudaSuccess) return e;
    q.rel_window = bias ? tc_rel_window(a) : 0;
    q.rel_part = (float *)(ws + w.part);
    q.rel_stride = q.rel_window ? (int)tc_rel_stride(a) : 0;
    const int heads = q.rel_window ? (int)tc_rel_heads(a) : pairs;
    float *rel = (float *)(ws + w.rel);
    for (int head0 = 0; head0 < pairs; head0 += heads) {
        const int now = std::min(heads, pairs - head0);
        q.head0 = head0;
        e = launch_attn_tc_bwd_kernel<T, false>(q, now, s);
        if (e != cudaSuccess) return e;
        if (q.rel_window)
            attn_rel_sum_kernel<<<dim3((a.R + 127) / 128, a.H), 128, 0, s>>>(
                a, q.rel_part, q.rel_stride, head0, now, rel);
    }
    *rel_done = q.rel_window > 0;
    return cudaGetLastError();
}

}  // namespace

template <typename T>
cudaError_t launch_attn(const AttnArgs &a, const AttnPtrs &p, void *ws, cudaStream_t s) {
    const float *bias = expand_bias<T>(a, p, ws, s);
    if constexpr (sizeof(T) == 2) {
        bool used = false;
        const cudaError_t e = launch_attn_tc_fwd<T>(a, p, bias, s, &used);
        if (used || e != cudaSuccess) return e;
    }
    attn_fwd_kernel<T><<<warp_blocks((int64_t)a.N * a.H * a.Lq), kWarps * 32, 0, s>>>(a, p, bias);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_attn_backward(const AttnArgs &a, const AttnPtrs &p, void *ws, cudaStream_t s) {
    const float *bias = expand_bias<T>(a, p, ws, s);
    const int threads = kWarps * 32;
    bool used = false, rel_done = false;
    if constexpr (sizeof(T) == 2) {
        const cudaError_t e = launch_tc_backward<T>(a, p, bias, (char *)ws, s, &used, &rel_done);
        if (e != cudaSuccess) return e;
    }
    if (!used) {
        attn_dq_kernel<T><<<warp_blocks((int64_t)a.N * a.H * a.Lq), threads, 0, s>>>(a, p, bias);
        attn_dkv_kernel<T><<<warp_blocks((int64_t)a.N * a.H * a.Lk), threads, 0, s>>>(a, p, bias);
    }
    if (a.nb) {
        float *rel = (float *)((char *)ws + workspace_of<T>(a, true).rel);
        if (!rel_done)
            attn_dbias_kernel<T><<<warp_blocks((int64_t)a.H * a.R), threads, 0, s>>>(a, p, bias, rel);
        attn_dtable_kernel<T><<<warp_blocks((int64_t)a.nb * a.H), threads, 0, s>>>(a, rel,
                                                                                  (T *)p.dTable);
    }
    return cudaGetLastError();
}

#define GS_ATTN_INST(T)                                                                         \
    template size_t attn_ws_bytes<T>(const AttnArgs &, bool);                                   \
    template cudaError_t launch_attn<T>(const AttnArgs &, const AttnPtrs &, void *, cudaStream_t); \
    template cudaError_t launch_attn_backward<T>(const AttnArgs &, const AttnPtrs &, void *,    \
                                                 cudaStream_t);
GS_ATTN_INST(float)
GS_ATTN_INST(__half)
GS_ATTN_INST(__nv_bfloat16)
#undef GS_ATTN_INST

}  // namespace gs
