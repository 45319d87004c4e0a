// gs_attn_few.cuh -- attention forward for few queries over many keys (a new
// token against a kept memory): every type, width and stride.
//
// The work is reading K and V once, so it is laid out for the loads: a key's
// row is read by a group of G lanes, 16 bytes each (or, where rows are not
// 16-byte aligned, by a whole warp, element by element), a batch of keys at a
// time with the next one in flight.  Each group keeps its own running maximum,
// sum and output for up to NQ queries; groups, warps and the blocks of a
// cluster, which share the keys of one head, are joined at the end (distributed
// shared memory: no second launch and no workspace).  The bias is looked up by
// one lane per key, the bucket two batches ahead and the entry one: looked up in
// place, the latency of both showed (130 us instead of 98).
//
// 8 x 8 heads, 32771 keys, D 64, bf16 (537 MB): 96.9 us, 5.5 TB/s, 0.82 of a copy's
// rate; 84.6 us where the lengths are between half and all of that (403 MB, 0.70),
// since the longest head sets the time.  One batch item: 24.4 us with clusters of
// up to sixteen blocks, 33.8 with eight.
#pragma once

#include <cooperative_groups.h>

#include "gs_attn_common.cuh"
#include "gs_ptx.cuh"

namespace gs {

constexpr int kFewThreads = 256;
constexpr int kFewMaxSplits = 16; // blocks of a cluster (more than 8: opted into)
constexpr int kFewLanes = 4;      // lanes of a key at least: a batch has no more keys than the warp lanes
constexpr int kFewQueries = 8;    // queries up to which this kernel is taken

// E consecutive (VEC: one 16-byte load) or 32-strided elements of a row.
template <typename T, bool VEC> struct FewRow {
    static constexpr int E = VEC ? 16 / sizeof(T) : 4;
    uint4 raw;
    float v[VEC ? 1 : E];
    __device__ __forceinline__ void load(const T *row, int part, int D, bool live) {
        if constexpr (VEC) {
            raw = make_uint4(0, 0, 0, 0);
            if (live && part * E < D) raw = __ldg(reinterpret_cast<const uint4 *>(row + part * E));
        } else {
#pragma unroll
            for (int k = 0; k < E; ++k)
                v[k] = live && part + 32 * k < D ? IO<T>::ld(row + part + 32 * k) : 0.0f;
        }
    }
    __device__ __forceinline__ float2 pair(int k) const { return make_float2(at(2 * k), at(2 * k + 1)); }
    __device__ __forceinline__ float at(int k) const {
        if constexpr (VEC) {
            const uint32_t *u = &raw.x;
            if constexpr (sizeof(T) == 4) {
                return __uint_as_float(u[k]);
            } else if constexpr (__is_same(T, __nv_bfloat16)) {
                return __uint_as_float(k % 2 ? u[k / 2] & 0xFFFF0000u : u[k / 2] << 16);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(u + k / 2));
                return k % 2 ? f.y : f.x;
            }
        } else {
            return v[k];
        }
    }
};

template <typename T, bool VEC, int NQ>
__global__ void __launch_bounds__(kFewThreads, 2)
    attn_few_kernel(AttnArgs a, AttnPtrs p, int G, int splits) {
    constexpr int E = FewRow<T, VEC>::E, W = kFewThreads / 32;
    constexpr int U = NQ == 1 ? 4 : 2;   // keys of a batch per group: what the registers hold
    __shared__ float s_o[W][NQ][128], s_m[W][NQ], s_l[W][NQ];   // per warp, then [0] per block
    const int groups = (a.Lq + NQ - 1) / NQ;
    const int64_t job = blockIdx.x / splits;
    const int rank = (int)(blockIdx.x % splits);
    const int i0 = (int)(job % groups) * NQ, h = (int)(job / groups % a.H);
    const int n = (int)(job / groups / a.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int part = lane % G, per_warp = 32 / G, group = lane / G;
    const float c2 = a.scale * kLog2e;
    const T *K = (const T *)p.K + n * a.ks[0] + h * a.ks[2];
    const T *V = (const T *)p.V + n * a.vs[0] + h * a.vs[2];
    const T *table = (const T *)p.table;

    float2 q[NQ][E / 2], o[NQ][E / 2];
    float m[NQ], l[NQ];
    int rq[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int i = min(i0 + x, a.Lq - 1);
        FewRow<T, VEC> r;
        r.load((const T *)p.Q + n * a.qs[0] + i * a.qs[1] + h * a.qs[2], part, a.D, true);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
            q[x][e] = make_float2(r.at(2 * e) * c2, r.at(2 * e + 1) * c2);
            o[x][e] = make_float2(0.0f, 0.0f);
        }
        m[x] = -INFINITY;
        l[x] = 0.0f;
        rq[x] = rel_q(a, i);
    }
    const int keys = keys_of(a, n);
    const int chunk = (keys + splits - 1) / splits;
    const int lo = min(rank * chunk, keys), hi = min(lo + chunk, keys);
    // The loads run ahead of their use: K, V and the bias by one batch of keys, the
    // buckets that name the bias by two.  A lane looks up the bias of one key of
    // the warp's batch, the groups get it from there.
    FewRow<T, VEC> k[U], v[U];
    T entry[NQ];              // table entries of the next batch
    int bucket[NQ];           // and the buckets of the batch after it, then of the next
    uint32_t has = 0;         // which of the entries there are, one bit per query
    const int batch = per_warp * U;   // 32 keys at most
    const auto load_buckets = [&](int base) {
        const int j = base + lane;
        const bool on = lane < batch && j < hi;
        const int rk = a.Hk == 1 ? j : on ? rel_k(a, j) : 0;
#pragma unroll
        for (int x = 0; x < NQ; ++x) bucket[x] = a.nb && on ? __ldg(a.buckets + rq[x] - rk) : -1;
    };
    const auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = base + u * per_warp + group;
            k[u].load(K + (int64_t)j * a.ks[1], part, a.D, j < hi);
            v[u].load(V + (int64_t)j * a.vs[1], part, a.D, j < hi);
        }
        has = 0;
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const bool in = (unsigned)bucket[x] < (unsigned)a.nb;
            entry[x] = in ? table[(int64_t)bucket[x] * a.H + h] : IO<T>::st(0.0f);
            if (a.nb ? in : base + lane < hi) has |= 1u << x;
        }
    };
    const int stride = W * batch;
    int base = lo + warp * batch;
    load_buckets(base);
    load(base);
    load_buckets(base + stride);
    for (; base < hi; base += stride) {
        float s[U][NQ], b[NQ];
        FewRow<T, VEC> keys_now[U], values[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            keys_now[u] = k[u];
            values[u] = v[u];
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x)
            b[x] = has >> x & 1 ? bias2(IO<T>::to_f(entry[x])) : -INFINITY;
        load(base + stride);
        load_buckets(base + 2 * stride);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) sum = fma_f32x2(q[x][e], keys_now[u].pair(e), sum);
                s[u][x] = sum.x + sum.y;
            }
        for (int w = G / 2; w > 0; w /= 2)
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int x = 0; x < NQ; ++x) s[u][x] += __shfl_xor_sync(0xffffffffu, s[u][x], w);
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float top = m[x];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                // a key that is not there stays masked whatever its score
                const float its = __shfl_sync(0xffffffffu, b[x], u * per_warp + group);
                s[u][x] = its == -INFINITY ? -INFINITY : s[u][x] + its;
                top = fmaxf(top, s[u][x]);
            }
            const float ref = top == -INFINITY ? 0.0f : top;
            const float keep = exp2_approx(m[x] - ref);
            m[x] = top;
            l[x] *= keep;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) o[x][e] = mul_f32x2(o[x][e], make_float2(keep, keep));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u][x] = exp2_approx(s[u][x] - ref);
                l[x] += s[u][x];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int x = 0; x < NQ; ++x)
#pragma unroll
                for (int e = 0; e < E / 2; ++e)
                    o[x][e] = fma_f32x2(make_float2(s[u][x], s[u][x]), values[u].pair(e), o[x][e]);
    }
    // join the groups of a warp
    for (int w = G; w < 32; w *= 2)
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[x], w);
            const float l2 = __shfl_xor_sync(0xffffffffu, l[x], w);
            const float top = fmaxf(m[x], m2), ref = top == -INFINITY ? 0.0f : top;
            const float f = exp2_approx(m[x] - ref), f2 = exp2_approx(m2 - ref);
            l[x] = l[x] * f + l2 * f2;
            m[x] = top;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float x2 = __shfl_xor_sync(0xffffffffu, o[x][e].x, w);
                const float y2 = __shfl_xor_sync(0xffffffffu, o[x][e].y, w);
                o[x][e] = make_float2(o[x][e].x * f + x2 * f2, o[x][e].y * f + y2 * f2);
            }
        }
    if (group == 0) {
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int d = VEC ? part * E + e : part + 32 * e;
                if (d < a.D) s_o[warp][x][d] = e % 2 ? o[x][e / 2].y : o[x][e / 2].x;
            }
            if (part == 0) {
                s_m[warp][x] = m[x];
                s_l[warp][x] = l[x];
            }
        }
    }
    __syncthreads();
    // join the warps of the block: a value per thread, into warp 0's place
    for (int at = threadIdx.x; at < NQ * a.D; at += kFewThreads) {
        const int x = at / a.D, d = at % a.D;
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][x]);
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < W; ++w) sum = fmaf(s_o[w][x][d], exp2_approx(s_m[w][x] - ref), sum);
        s_o[0][x][d] = sum;
    }
    __syncthreads();
    if (threadIdx.x < NQ) {
        const int x = threadIdx.x;
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][x]);
        const float ref = top == -INFINITY ? 0.0f : top;
        for (int w = 0; w < W; ++w) sum = fmaf(s_l[w][x], exp2_approx(s_m[w][x] - ref), sum);
        s_m[0][x] = top;
        s_l[0][x] = sum;
    }
    // join the blocks of the cluster
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (splits > 1)
        cluster.sync();
    else
        __syncthreads();
    if (rank == 0) {
        for (int at = threadIdx.x; at < NQ * a.D; at += kFewThreads) {
            const int x = at / a.D, d = at % a.D;
            if (i0 + x >= a.Lq) break;
            float top = -INFINITY, sum = 0.0f, l_all = 0.0f;
            for (int r = 0; r < splits; ++r)
                top = fmaxf(top, splits > 1 ? *cluster.map_shared_rank(&s_m[0][x], r) : s_m[0][x]);
            const float ref = top == -INFINITY ? 0.0f : top;
            for (int r = 0; r < splits; ++r) {
                const float mr = splits > 1 ? *cluster.map_shared_rank(&s_m[0][x], r) : s_m[0][x];
                const float lr = splits > 1 ? *cluster.map_shared_rank(&s_l[0][x], r) : s_l[0][x];
                const float v = splits > 1 ? *cluster.map_shared_rank(&s_o[0][x][d], r) : s_o[0][x][d];
                const float f = exp2_approx(mr - ref);
                sum = fmaf(v, f, sum);
                l_all = fmaf(lr, f, l_all);
            }
            ((T *)p.O)[(((int64_t)n * a.Lq + i0 + x) * a.H + h) * a.D + d] =
                IO<T>::st(l_all != 0.0f ? sum / l_all : 0.0f);
            if (d == 0 && p.lse)
                p.lse[((int64_t)n * a.H + h) * a.Lq + i0 + x] = lse_of(top, l_all);
        }
    }
    if (splits > 1) cluster.sync();   // shared memory stays until rank 0 has read it
}

inline bool few_takes(const AttnArgs &a) { return a.Lq <= kFewQueries; }

// splits: blocks per head, as many as the SMs hold at once with two each (a
// second wave would leave most of them idle), of at least 128 keys.
template <typename T, bool VEC, int NQ>
cudaError_t launch_attn_few_as(const AttnArgs &a, const AttnPtrs &p, int G, cudaStream_t s) {
    const int64_t jobs = (int64_t)((a.Lq + NQ - 1) / NQ) * a.H * a.N;
    int splits = 1;
    while (splits < kFewMaxSplits && jobs * splits * 2 <= 152 * 2 && a.Lk > 128 * splits) splits *= 2;
    static DeviceFlags ready;
    const cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(attn_few_kernel<T, VEC, NQ>,
                                    cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(jobs * splits));
    cfg.blockDim = dim3(kFewThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, attn_few_kernel<T, VEC, NQ>, a, p, G, splits);
}

template <typename T>
cudaError_t launch_attn_few(const AttnArgs &a, const AttnPtrs &p, cudaStream_t s) {
    constexpr int E = 16 / sizeof(T);
    bool vec = a.D % E == 0;
    for (const void *x : {p.Q, p.K, p.V}) vec = vec && ((uintptr_t)x & 15u) == 0;
    for (int d = 0; d < 3; ++d)
        vec = vec && a.qs[d] % E == 0 && a.ks[d] % E == 0 && a.vs[d] % E == 0;
    int G = 32;   // lanes per key: a power of two that covers the row, kFewLanes at least
    if (vec)
        while (G > kFewLanes && G / 2 * E >= a.D) G /= 2;
    if (vec)
        return a.Lq == 1 ? launch_attn_few_as<T, true, 1>(a, p, G, s)
                         : launch_attn_few_as<T, true, 4>(a, p, G, s);
    return a.Lq == 1 ? launch_attn_few_as<T, false, 1>(a, p, G, s)
                     : launch_attn_few_as<T, false, 4>(a, p, G, s);
}

}  // namespace gs
