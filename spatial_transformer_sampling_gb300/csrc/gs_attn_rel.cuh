// gs_attn_rel.cuh -- the gradient of the bias by relative index, and the row
// sums both backward paths start from.
//
// For one column (key) the relative indices of a warp's rows
// are all different, so each warp adds ds to a private window in shared memory
// without atomics, four columns at a time in four copies.  Going along the
// keys the window moves down; indices above it are final and are written once
// per warp to `part`, which attn_rel_sum_kernel adds up in a fixed order.
#pragma once

#include <algorithm>

#include "gs_attn_common.cuh"

namespace gs {

constexpr int kRelCopies = 4;
constexpr int kRelCols = 64;      // keys of one step

// Where a launch of the query kernel leaves its share of the bias gradient.
struct RelArgs {
    int window;     // floats of a warp's window, a power of two (0: not computed there)
    int stride;     // floats a query warp writes
    int head0;      // first (batch, head) pair of the launch
    float *part;    // (pairs of the launch, query warps, stride)
};

// Rows of lse2 and delta kept per (batch, head): whole column tiles.
__host__ __device__ inline int rows64(int L) { return (L + 63) / 64 * 64; }

// Shared memory of `warps` bias-gradient windows of `w` floats: per warp four
// copies, the moving window and the columns' relative indices.
inline __host__ __device__ int rel_smem(int w, int warps) {
    return w ? warps * ((kRelCopies + 1) * w + kRelCols) * 4 : 0;
}

// Adds one step's ds (fp32, 64 columns of this thread's query) to the warp's
// bias-gradient window and writes out the indices that are final.
struct RelWindow {
    float *copies, *ring;
    int *rel;
    int size, rq, rq_min, rq_max, top;
    bool mine;

    // Warp `threadIdx.x / 32` of the block takes queries i0 + 32 * warp on, of the
    // (batch, head) pair nh.  Returns where it writes, indexed by relative index.
    __device__ __forceinline__ float *init(const AttnArgs &a, float *smem, const RelArgs &p, int i0,
                                           int nh) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, iw = i0 + warp * 32;
        size = p.window;
        copies = smem + warp * ((kRelCopies + 1) * size + kRelCols);
        ring = copies + kRelCopies * size;
        rel = reinterpret_cast<int *>(ring + size);
        for (int k = lane; k < (kRelCopies + 1) * size; k += 32) copies[k] = 0.0f;
        mine = iw + lane < a.Lq;
        rq = rel_q(a, min(iw + lane, a.Lq - 1));
        rq_min = rel_q(a, min(iw, a.Lq - 1));
        rq_max = rel_q(a, min(iw + 31, a.Lq - 1));
        top = rq_max;
        __syncwarp();
        const int64_t slot = (int64_t)(nh - p.head0) * ((a.Lq + 31) / 32) + iw / 32;
        return p.part + slot * p.stride - (rq_min - rel_k(a, a.Lk - 1));
    }

    // keys j0 .. j0 + live - 1 of `keys`; `out` is indexed by relative index
    __device__ __forceinline__ void add(const AttnArgs &a, const float (&ds)[kRelCols], int j0, int live,
                                        int keys, float *out) {
        const int lane = threadIdx.x % 32;
        live = min(live, kRelCols);
#pragma unroll
        for (int k = 0; k < kRelCols; k += 32) rel[k + lane] = rel_k(a, min(j0 + k + lane, keys - 1));
        __syncwarp();
        const int lo = rq_min - rel[live - 1];
        const int span = rq_max - rel[0] - lo + 1;
        float *at = copies + (rq - lo);
#pragma unroll
        for (int s = 0; s < kRelCols / kRelCopies; ++s) {
            float v[kRelCopies];
            int k[kRelCopies];
#pragma unroll
            for (int g = 0; g < kRelCopies; ++g) {
                const int c = s + g * (kRelCols / kRelCopies);
                k[g] = g * size - rel[c];
                if (c < live && mine) v[g] = at[k[g]] + ds[c];
            }
#pragma unroll
            for (int g = 0; g < kRelCopies; ++g)
                if (s + g * (kRelCols / kRelCopies) < live && mine) at[k[g]] = v[g];
            __syncwarp();
        }
        // join the copies into the ring, which is indexed by the relative index
        for (int k = lane; k < span; k += 32) {
            float v = 0.0f;
#pragma unroll
            for (int g = 0; g < kRelCopies; ++g) {
                v += copies[g * size + k];
                copies[g * size + k] = 0.0f;
            }
            ring[(lo + k) & (size - 1)] += v;
        }
        __syncwarp();
        const int final_above = j0 + live < keys ? rq_max - rel_k(a, j0 + live) : lo - 1;
        for (int r = final_above + 1 + lane; r <= top; r += 32) {
            out[r] = ring[r & (size - 1)];
            ring[r & (size - 1)] = 0.0f;
        }
        top = final_above;
        __syncwarp();
    }
};

// lse2 and delta of every query, sixteen threads per row (VEC: 16-bit types,
// 16-byte rows).
template <typename T, bool VEC>
__global__ void attn_delta_kernel(AttnArgs a, const T *dO, const T *O, const float *lse,
                                  float *lse2, float *delta) {
    const int L64 = rows64(a.Lq), part = threadIdx.x % 16;
    const int64_t row = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 16;   // (n, i, h)
    if (row >= (int64_t)a.N * L64 * a.H) return;
    const int h = (int)(row % a.H), i = (int)(row / a.H % L64), n = (int)(row / a.H / L64);
    float s = 0.0f;
    const int64_t at = (((int64_t)n * a.Lq + i) * a.H + h) * a.D;
    if (!VEC) {
        if (i < a.Lq)
            for (int d = part; d < a.D; d += 16) s = fmaf(IO<T>::ld(dO + at + d), IO<T>::ld(O + at + d), s);
    } else if (i < a.Lq && part * 8 < a.D) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(dO + at + part * 8));
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(O + at + part * 8));
        const T *x = reinterpret_cast<const T *>(&u), *y = reinterpret_cast<const T *>(&v);
#pragma unroll
        for (int k = 0; k < 16 / (int)sizeof(T); ++k) s = fmaf(IO<T>::to_f(x[k]), IO<T>::to_f(y[k]), s);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (part == 0) {
        const int64_t nh = (int64_t)n * a.H + h;
        const float v = i < a.Lq ? lse[nh * a.Lq + i] : -INFINITY;
        lse2[nh * L64 + i] = v == -INFINITY ? INFINITY : v * kLog2e;   // no key: weights of 0
        delta[nh * L64 + i] = s;
    }
}

// rel[h][r] (+)= the warps' sums, query warps and batch items in a fixed order;
// `heads` (batch, head) pairs from head0 on are in `part`.
static __global__ void attn_rel_sum_kernel(AttnArgs a, RelArgs p, int heads, float *rel) {
    constexpr int kThreads = 128;
    __shared__ int s_lo[kThreads], s_hi[kThreads];   // relative indices of a warp's queries
    const int r = blockIdx.x * kThreads + threadIdx.x, h = blockIdx.y;
    const int warps = (a.Lq + 31) / 32, k_end = rel_k(a, a.Lk - 1);
    float sum = p.head0 > 0 && r < a.R ? rel[(int64_t)h * a.R + r] : 0.0f;
    for (int w0 = 0; w0 < warps; w0 += kThreads) {
        const int mine = min(w0 + (int)threadIdx.x, warps - 1);
        __syncthreads();
        s_lo[threadIdx.x] = rel_q(a, mine * 32);
        s_hi[threadIdx.x] = rel_q(a, min(mine * 32 + 31, a.Lq - 1));
        __syncthreads();
        const int count = min(kThreads, warps - w0);
        for (int nh = p.head0 + (h - p.head0 % a.H + a.H) % a.H; nh < p.head0 + heads; nh += a.H) {
            const int keys = keys_of(a, nh / a.H);
            const int low = keys > 0 ? rel_k(a, keys - 1) : -1;   // of r below the queries' lowest
            const float *at = p.part + ((int64_t)(nh - p.head0) * warps + w0) * p.stride + r + k_end;
#pragma unroll 8
            for (int w = 0; w < count; ++w)
                if (keys > 0 && r <= s_hi[w] && r >= s_lo[w] - low)
                    sum += __ldg(at + (int64_t)w * p.stride - s_lo[w]);
        }
    }
    if (r < a.R) rel[(int64_t)h * a.R + r] = sum;
}

// Relative indices between the first and the last of `tokens` consecutive
// tokens of a grid of `rows` rows of W, at most: one per token and P - W more
// at each end of a grid row.
inline int64_t rel_span(int tokens, int L, int rows, int W, int P) {
    const int64_t t = std::min(tokens, L) - 1;
    const int64_t crossings = t <= 0 ? 0 : std::min<int64_t>((t - 1) / W + 1, rows - 1);
    return t + crossings * (P - W);
}

// Power of two that holds the relative indices of a warp's 32 queries against
// 64 keys; 0 when that is more than 1024 (rows of hundreds of tokens that end
// inside a tile): 20 KB of windows per 256 floats.
inline int rel_window_of(const AttnArgs &a) {
    const int64_t span = rel_span(32, a.Lq, a.Hq, a.Wq, a.P) + rel_span(kRelCols, a.Lk, a.Hk, a.Wk, a.P) + 1;
    int w = 128;
    while (w < span) w *= 2;
    return w <= 1024 ? w : 0;
}
// Floats a query warp writes to `part`.
inline int64_t rel_stride_of(const AttnArgs &a) {
    return rel_span(32, a.Lq, a.Hq, a.Wq, a.P) + (int64_t)(a.Hk - 1) * a.P + a.Wk;
}
// (batch, head) pairs of one launch: all, or as many as keep `part` within
// 256 MB (one at least); their sums are added launch by launch.
inline int64_t rel_heads_of(const AttnArgs &a) {
    const int64_t per = (int64_t)((a.Lq + 31) / 32) * rel_stride_of(a) * 4;
    return std::max<int64_t>(1, std::min<int64_t>((int64_t)a.N * a.H, (int64_t(256) << 20) / per));
}

}  // namespace gs
