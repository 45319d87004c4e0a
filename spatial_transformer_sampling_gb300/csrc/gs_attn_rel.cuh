// gs_attn_rel.cuh -- the gradient of the bias by relative index, and the row
// sums both backward paths start from.
//
// For one column (key) the relative indices of 32 queries are all different, so
// a warp adds ds to a window in shared memory without atomics.  Two warps share
// 32 queries, half of a step's 64 keys each, two columns at a time in a copy
// of its own each (four copies).  Going along the keys the window moves down;
// indices above it are final and are written once per 32 queries to `part`,
// which attn_rel_sum_kernel adds up in a fixed order.
#pragma once

#include <limits.h>

#include <algorithm>

#include "gs_attn_common.cuh"
#include "gs_ptx.cuh"

namespace gs {

constexpr int kRelCopies = 4;     // two for each of the two warps
constexpr int kRelCols = 64;      // keys of one step
constexpr int kRelHalf = kRelCols / 2;
constexpr int kRelMost = 1024;    // floats of the largest window

// Where a launch of the query kernel leaves its share of the bias gradient.
struct RelArgs {
    int window;     // floats of a window, a power of two (0: not computed there)
    int stride;     // floats written per 32 queries
    int head0;      // first (batch, head) pair of the launch
    float *part;    // (pairs of the launch, groups of 32 queries, stride)
};

// Rows of lse2 and delta kept per (batch, head): whole column tiles.
__host__ __device__ inline int rows64(int L) { return (L + 63) / 64 * 64; }

// Shared memory of `pairs` bias-gradient windows of `w` floats: four copies, the
// moving window and the columns' relative indices each.
inline __host__ __device__ constexpr int rel_smem(int w, int pairs) {
    return w ? pairs * ((kRelCopies + 1) * w + kRelCols) * 4 : 0;
}

// The window of 32 queries, held by a pair of warps (`half` 0 and 1).
struct RelWindow {
    float *copies, *ring;
    int *rel;
    int size, rq, rq_min, rq_max, top, pair, half;
    bool mine;

    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
    }

    // The pair takes queries i0 + 32 * pair on of the (batch, head) pair nh.
    // Returns where it writes, indexed by relative index.
    __device__ __forceinline__ float *init(const AttnArgs &a, float *smem, const RelArgs &p, int i0,
                                           int nh, int pair_, int half_) {
        pair = pair_;
        half = half_;
        const int lane = threadIdx.x % 32, iw = i0 + pair * 32;
        size = p.window;
        copies = smem + pair * ((kRelCopies + 1) * size + kRelCols);
        ring = copies + kRelCopies * size;
        rel = reinterpret_cast<int *>(ring + size);
        for (int k = half * 32 + lane; k < (kRelCopies + 1) * size; k += 64) copies[k] = 0.0f;
        mine = iw + lane < a.Lq;
        rq = rel_q(a, min(iw + lane, a.Lq - 1));
        rq_min = rel_q(a, min(iw, a.Lq - 1));
        rq_max = rel_q(a, min(iw + 31, a.Lq - 1));
        top = rq_max;
        const int64_t slot = (int64_t)(nh - p.head0) * ((a.Lq + 31) / 32) + iw / 32;
        return p.part + slot * p.stride - (rq_min - rel_k(a, a.Lk - 1));
    }

    // ds (fp32) of this thread's query and its half of a step's 64 keys, of which
    // `live` count.  my_rel: rel_k of key half * 32 + lane of the step (of the last
    // live one from there on); next_rel: of the next step's first key (`last`:
    // there is none).  Both warps call it; `out` as from init.
    __device__ __forceinline__ void add(const float (&ds)[kRelHalf], int live, int my_rel,
                                        int next_rel, bool last, float *out) {
        const int lane = threadIdx.x % 32, first = half * kRelHalf;
        live = min(live, kRelCols);
        rel[first + lane] = my_rel;
        const bool all = __all_sync(0xffffffffu, mine);
        sync();   // and the windows are clear
        const int lo = rq_min - rel[live - 1];
        const int span = rq_max - rel[0] - lo + 1;
        float *at = copies + 2 * half * size + (rq - lo);
        constexpr int kStep = kRelHalf / 2;
        if (all && live == kRelCols && rel[first + kRelHalf - 1] - rel[first] == kRelHalf - 1) {
            // all rows and columns count and the columns are neighbours in a grid row
            float *p0 = at - rel[first], *p1 = p0 + size - kStep;
#pragma unroll
            for (int s = 0; s < kStep; ++s) {
                const float v0 = p0[-s] + ds[s], v1 = p1[-s] + ds[kStep + s];
                p0[-s] = v0;
                p1[-s] = v1;
                __syncwarp();
            }
        } else {
#pragma unroll
            for (int s = 0; s < kStep; s += 4) {
                const int4 o0 = *reinterpret_cast<const int4 *>(rel + first + s);
                const int4 o1 = *reinterpret_cast<const int4 *>(rel + first + kStep + s);
                const int k0[4] = {o0.x, o0.y, o0.z, o0.w}, k1[4] = {o1.x, o1.y, o1.z, o1.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool on0 = mine && first + s + e < live;
                    const bool on1 = mine && first + kStep + s + e < live;
                    float v0, v1;
                    if (on0) v0 = at[-k0[e]] + ds[s + e];
                    if (on1) v1 = at[size - k1[e]] + ds[kStep + s + e];
                    if (on0) at[-k0[e]] = v0;
                    if (on1) at[size - k1[e]] = v1;
                    __syncwarp();
                }
            }
        }
        sync();
        // join the copies into the ring, which is indexed by the relative index
        for (int k = half * 32 + lane; k < span; k += 64) {
            float v = 0.0f;
#pragma unroll
            for (int g = 0; g < kRelCopies; ++g) {
                v += copies[g * size + k];
                copies[g * size + k] = 0.0f;
            }
            ring[(lo + k) & (size - 1)] += v;
        }
        sync();
        const int final_above = last ? lo - 1 : rq_max - next_rel;
        for (int r = final_above + 1 + half * 32 + lane; r <= top; r += 64) {
            out[r] = ring[r & (size - 1)];
            ring[r & (size - 1)] = 0.0f;
        }
        top = final_above;
    }
};

// How far dS may be scaled up on its way to a 16-bit type: the largest sums of
// squares of a dO row and of a live V row, in `parts` shares per (batch, head)
// pair.  By Cauchy and Schwarz their product bounds dP, and delta, in which V is
// averaged, as well.  Rows that are not finite do not count: what they reach is
// not finite either way.
struct RangeArgs {
    int parts;      // 0: not wanted
    float *most;    // (pairs, parts, 2): dO, V
};
constexpr int kRangeMost = 32;     // shares at most, one per lane of the warps that read them
constexpr int kRangeRows = 64;     // rows of a share at least: two batches of loads at D = 64
inline int range_parts(const AttnArgs &a) {
    return std::min((std::max(a.Lq, a.Lk) + kRangeRows - 1) / kRangeRows, kRangeMost);
}

// One share: `part` of dO's and V's rows, which are runs of 16 bytes.
template <typename T>
__device__ __forceinline__ void attn_range_block(const AttnArgs &a, const T *dO, const T *V,
                                                 const RangeArgs &range, int block) {
    constexpr int E = 16 / (int)sizeof(T);
    __shared__ float s_most[8];
    const int nh = block / range.parts, part = block % range.parts, n = nh / a.H, h = nh % a.H;
    int G = 1;   // lanes of a row
    while (G * E < a.D) G *= 2;
    const int lane = threadIdx.x % G;
    for (int which = 0; which < 2; ++which) {
        const int rows = which ? keys_of(a, n) : a.Lq;
        const int64_t step = which ? a.vs[1] : (int64_t)a.H * a.D;
        const T *base = which ? V + n * a.vs[0] + h * a.vs[2] : dO + ((int64_t)n * a.Lq * a.H + h) * a.D;
        const int chunk = (rows + range.parts - 1) / range.parts;
        const int end = min((part + 1) * chunk, rows);
        float most = 0.0f;
#pragma unroll 4
        for (int r0 = part * chunk; r0 < end; r0 += 256 / G) {   // the same for all threads
            const int r = r0 + threadIdx.x / G;
            float sum = 0.0f;
            if (r < end && lane * E < a.D) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(base + r * step + lane * E));
                const T *x = reinterpret_cast<const T *>(&u);
#pragma unroll
                for (int k = 0; k < E; ++k) sum = fmaf(IO<T>::to_f(x[k]), IO<T>::to_f(x[k]), sum);
            }
            for (int o = G / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (sum < INFINITY) most = fmaxf(most, sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        __syncthreads();
        if (threadIdx.x % 32 == 0) s_most[threadIdx.x / 32] = most;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < 8; ++w) most = fmaxf(most, s_most[w]);
            range.most[((int64_t)nh * range.parts + part) * 2 + which] = most;
        }
    }
}

// lse2 and delta of every query (6.6 us for the 17 MB of 8 x 8 heads of 32 x 32
// tokens, D 64, bf16: latency and memory; 12 us in fp16 with RANGE), G lanes per row (a
// power of two; VEC: rows of 16-byte runs, one per lane).  A block takes 256 / G rows
// of one batch item, in memory order (token, head).  RANGE: the blocks behind those
// take a share of RangeArgs each.
template <typename T, bool VEC, bool RANGE>
__global__ void attn_delta_kernel(AttnArgs a, const T *dO, const T *O, const T *V, const float *lse,
                                  int G, int blocks_per_item, float *lse2, float *delta,
                                  RangeArgs range) {
    constexpr int E = 16 / (int)sizeof(T);
    const int row_blocks = blocks_per_item * a.N;
    if (RANGE && (int)blockIdx.x >= row_blocks) {
        attn_range_block(a, dO, V, range, blockIdx.x - row_blocks);
        wait_for_previous_kernel();
        return;
    }
    const int L64 = rows64(a.Lq), part = threadIdx.x % G;
    const int n = blockIdx.x / blocks_per_item;
    const int64_t row = (int64_t)(blockIdx.x % blocks_per_item) * (256 / G) + threadIdx.x / G;
    const int i = (int)(row / a.H), h = (int)(row - (int64_t)i * a.H);
    float s = 0.0f;
    if (i < a.Lq) {
        const int64_t at = ((int64_t)n * a.Lq * a.H + row) * a.D;
        if (!VEC) {
            for (int d = part; d < a.D; d += G) s = fmaf(IO<T>::ld(dO + at + d), IO<T>::ld(O + at + d), s);
        } else if (part * E < a.D) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(dO + at + part * E));
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(O + at + part * E));
            const T *x = reinterpret_cast<const T *>(&u), *y = reinterpret_cast<const T *>(&v);
#pragma unroll
            for (int k = 0; k < E; ++k) s = fmaf(IO<T>::to_f(x[k]), IO<T>::to_f(y[k]), s);
        }
    }
    for (int o = G / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (part == 0 && i < L64) {
        const int64_t nh = (int64_t)n * a.H + h;
        const float v = i < a.Lq ? lse[nh * a.Lq + i] : -INFINITY;
        lse2[nh * L64 + i] = lse2_of(v);
        delta[nh * L64 + i] = s;
    }
    // nothing here reads the expanded bias, but the kernels that wait for this
    // one's end do
    wait_for_previous_kernel();
}

template <typename T>
cudaError_t launch_attn_delta(const AttnArgs &a, const AttnPtrs &p, float *lse2, float *delta,
                              const RangeArgs &range, cudaStream_t s) {
    constexpr int E = 16 / (int)sizeof(T);
    const bool vec = a.D % E == 0 && (((uintptr_t)p.dO | (uintptr_t)p.O) & 15u) == 0;
    int G = vec ? 1 : 16;
    while (vec && G * E < a.D) G *= 2;
    const int64_t per_item = ((int64_t)rows64(a.Lq) * a.H * G + 255) / 256;
    auto kernel = vec ? attn_delta_kernel<T, true, false> : attn_delta_kernel<T, false, false>;
    if constexpr (__is_same(T, __half))   // its rows are then runs of 16 bytes
        if (range.parts) kernel = attn_delta_kernel<T, true, true>;
    return launch_next(a.nb > 0, kernel, (unsigned)(per_item * a.N + (int64_t)a.N * a.H * range.parts), 256,
                       0, s, a, (const T *)p.dO, (const T *)p.O, (const T *)p.V, p.lse, G, (int)per_item,
                       lse2, delta, range);
}

// Groups of 32 queries whose sums attn_rel_sum_kernel goes through at a time: as
// many as threads, fewer where their offsets from the first one, `stride` floats a
// group, would not fit 32 bits beside two relative indices (which stay below 2^25).
// 512 groups of 16384 queries over 4 M keys would be 2^31.
constexpr int kRelSumThreads = 512;
__host__ __device__ inline int rel_groups_at_once(int stride) {
    const int most = (1 << 30) / stride;
    return most < kRelSumThreads ? most : kRelSumThreads;
}

// rel[h][r] (+)= the sums of groups of 32 queries; `heads` (batch, head) pairs
// from head0 on are in `part`.  128 indices a block, four per thread; sixteen
// warps take every sixteenth (item, group) pair and are joined in order.  Bound by
// the latency of the loads: 8 x 8 heads of 32 x 32 tokens (16 MB, in L2) take 8.9 us,
// 16.5 with eight warps and 11.3 with 32, which fewer SMs hold at a time.
constexpr int kRelSumIndices = 128;
static __global__ void __launch_bounds__(kRelSumThreads)
    attn_rel_sum_kernel(AttnArgs a, RelArgs p, int heads, float *rel) {
    constexpr int kSlices = kRelSumThreads / 32, kChunk = kRelSumThreads, kEach = kRelSumIndices / 32;
    // per group of queries: its lowest and highest relative index, and where its
    // entry 0 lies from the first group's sums; per item: those of the first group, and
    // how far the relative indices reach below a group's lowest one
    __shared__ int s_lo[kChunk], s_hi[kChunk], s_at[kChunk], s_low[kChunk];
    __shared__ const float *s_item[kChunk];
    __shared__ float s_sum[kSlices][kRelSumIndices];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32;
    const int r = blockIdx.x * kRelSumIndices + lane, h = blockIdx.y;
    const int groups = (a.Lq + 31) / 32, k_end = rel_k(a, a.Lk - 1);
    const int nh0 = p.head0 + (h - p.head0 % a.H + a.H) % a.H;   // this head's first pair
    const int items = nh0 < p.head0 + heads ? (p.head0 + heads - 1 - nh0) / a.H + 1 : 0;
    const int at_once = rel_groups_at_once(p.stride);
    float sum[kEach] = {};
    wait_for_previous_kernel(p.part, rel);
    for (int n0 = 0; n0 < items; n0 += kChunk)
        for (int w0 = 0; w0 < groups; w0 += at_once) {
            const int w_mine = min(w0 + min((int)threadIdx.x, at_once - 1), groups - 1);
            const int nh = nh0 + min(n0 + (int)threadIdx.x, items - 1) * a.H;
            const int keys = keys_of(a, nh / a.H);
            __syncthreads();
            s_lo[threadIdx.x] = rel_q(a, w_mine * 32);
            s_hi[threadIdx.x] = rel_q(a, min(w_mine * 32 + 31, a.Lq - 1));
            s_at[threadIdx.x] = (w_mine - w0) * p.stride + k_end - s_lo[threadIdx.x];
            s_item[threadIdx.x] = p.part + ((int64_t)(nh - p.head0) * groups + w0) * p.stride;
            s_low[threadIdx.x] = keys > 0 ? rel_k(a, keys - 1) : INT_MIN / 2;
            __syncthreads();
            const int nw = min(at_once, groups - w0), nn = min(kChunk, items - n0);
            int i = slice / nw, w = slice % nw;
            const int di = kSlices / nw, dw = kSlices % nw;
#pragma unroll 4
            for (int k = slice; k < nn * nw; k += kSlices) {
                const int hi = s_hi[w], lo = s_lo[w] - s_low[i];
                const float *at = s_item[i] + s_at[w] + r;
#pragma unroll
                for (int q = 0; q < kEach; ++q)
                    if (r + 32 * q <= hi && r + 32 * q >= lo) sum[q] += __ldg(at + 32 * q);
                i += di;
                w += dw;
                if (w >= nw) {
                    w -= nw;
                    ++i;
                }
            }
        }
#pragma unroll
    for (int q = 0; q < kEach; ++q) s_sum[slice][lane + 32 * q] = sum[q];
    __syncthreads();
    for (int k = threadIdx.x; k < kRelSumIndices; k += kRelSumThreads) {
        const int at = blockIdx.x * kRelSumIndices + k;
        float all = 0.0f;
        for (int w = 0; w < kSlices; ++w) all += s_sum[w][k];
        if (at < a.R) {
            float *out = rel + (int64_t)h * a.R + at;
            *out = p.head0 > 0 ? *out + all : all;
        }
    }
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
// 64 keys, and those that become final before the next 64: the distance to the
// next step's first key may cross one grid row more than a step's keys do (rows of
// 63 tokens, from the last of one on).  0 when that is more than kRelMost (rows of
// hundreds of tokens that end inside a tile): 20 KB of windows per 256 floats.
inline int rel_window_of(const AttnArgs &a) {
    const int64_t span = rel_span(32, a.Lq, a.Hq, a.Wq, a.P) +
                         rel_span(kRelCols + 1, a.Lk, a.Hk, a.Wk, a.P) + 1;
    int w = 128;
    while (w < span) w *= 2;
    return w <= kRelMost ? w : 0;
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
