// gs_attn_tc_fwd.cuh -- attention forward on the tensor cores (fp16 / bf16).
//
// One CTA per 128 queries of one head, two to an SM; it walks the keys 64 at a time:
//   S = Q K^T             tcgen05.mma, fp32 in TMEM, two buffers
//   p = 2^(c S + bias - m)  two softmax threads per query, m its running reference
//   O += p V              tcgen05.mma with p (16-bit) read from TMEM, where it
//                         overwrites the scores it came from
// so scores and weights never leave the SM.  The two threads of a query take 32
// keys each and exchange their maxima through shared memory.  One thread of a
// ninth warp issues the MMAs (the scores of tile j + 1 are computed while the
// softmax warps work on tile j), one of a tenth the TMA loads: issued by one
// warp with votes between, both took longer than the softmax.  Where heads are
// short a CTA goes through several items of 128 queries (kFwdMany): the copies and
// the scores of the next one run ahead of the end of the current one, whose
// output is stored after the next one's first tile.
//
// Bound by the softmax warps, their instructions (58 % of the issue slots) and the
// latency of the exchange through TMEM; the tensor pipe is busy 20 %.  8 x 8 heads
// of 64 x 64 tokens, D 64, fp16, with bias: 470 us, 585 TFLOP/s (0.30 of a large
// matrix product's rate).
//
// Running maximum and sum as in Milakov and Gimelshein, "Online normalizer
// calculation for softmax" (2018), but that the reference m follows the maximum
// lazily: O and the row sum are rescaled only when it has grown by more than 2^8
// since (the final division cancels m; weights stay below 2^8, inside both 16-bit
// types).  The row sum is kept in fp32 from the unrounded weights.  The weights are
// rounded to T, since the matrix instruction takes both operands in one 16-bit type:
// half a step of T on every term, with the store 2.0e-3 of O in bf16 (windows) and
// 2.9e-4 in fp16 (64 x 64 tokens), against 1.7e-3 and 2.1e-4 for the store alone.
//
// The bias of a tile comes to shared memory with the keys (TcBias).
#pragma once

#include <cooperative_groups.h>

#include "gs_attn_tc.cuh"

namespace gs {

struct TcFwdArgs {
    AttnArgs a;
    TcView q, k, v;
    TcBias bias;
    void *O;
    float *lse;
};

constexpr int kTcSms = 152;
constexpr float kLazyGrowth = 8.0f;   // log2 of how far the maximum may outgrow the reference

// log2 of the weight at the reference: fp16 weights are kept 2^6 up, so that
// small ones stay clear of the type's subnormal range (2^14 at most).
template <typename T> constexpr float kWeightShift = 0.0f;
template <> constexpr float kWeightShift<__half> = 6.0f;

// How blocks and items of 128 queries go together: a block each, a block for
// several items (short heads), a cluster for one (few items of long heads).
enum { kFwdOne = 0, kFwdMany = 1, kFwdSplit = 2 };

template <int DP, int MODE> struct TcFwdShape {
    static constexpr bool MANY = MODE == kFwdMany;
    static constexpr int kStages = DP == 64 ? 3 : 2;
    // queries and outputs of two items at a time, where both fit
    static constexpr int kItems = MANY && DP == 64 ? 2 : 1;
    static constexpr int kQBytes = kTcM * DP * 2;
    static constexpr int kTileBytes = kTcN * DP * 2;
    static constexpr int kTileSmem = kItems * kQBytes + 2 * kStages * kTileBytes;
    static constexpr int kSmem = kTileSmem + 1024;   // 1024-byte alignment of the tiles
    static constexpr int kTmemCols = 256;            // two score buffers, O; two CTAs per SM
    static constexpr int kTmemO = 2 * kTcN;
    // a block's share of the output, over the tiles, for the other blocks of the cluster
    static constexpr int kSharePitch = DP + 4;
    static_assert(MODE != kFwdSplit || kTcM * kSharePitch * 4 <= kTileSmem, "fits the tiles");
};

// An item of work: 128 queries of one head.  A CTA takes one, or with kFwdMany every
// gridDim.x-th one, or with kFwdSplit its part of one's keys; its key tiles are
// numbered through (`tile`), which gives a tile its score buffer, its stage of NS and the parity of their barriers' phases, and so are
// the items that have keys (`count`).
template <int NS, int MODE> struct TcItem {
    static constexpr bool MANY = MODE == kFwdMany;
    // key0: the first key that is taken, `keys` how many from there on
    int index, n, h, i0, key0, keys, tiles, j, tile, stage, parity, count;
    __device__ __forceinline__ void decode(const AttnArgs &a, int q_tiles) {
        i0 = index % q_tiles * kTcM;
        h = index / q_tiles % a.H;
        n = index / q_tiles / a.H;
        keys = keys_of(a, n);
        tiles = (keys + kTcN - 1) / kTcN;
        key0 = 0;
        if (MODE == kFwdSplit) {   // whole tiles each, the last ones fewer or none
            const int share = (tiles + cluster_size() - 1) / cluster_size();
            const int first = min(cluster_rank() * share, tiles);
            tiles = min(share, tiles - first);
            key0 = first * kTcN;
            keys = min(keys - key0, tiles * kTcN);
        }
    }
    // The first item with keys from `index` on; false when there is none.
    __device__ __forceinline__ bool seek(const AttnArgs &a, int q_tiles, int items) {
        for (; index < items; index += gridDim.x) {
            decode(a, q_tiles);
            if (tiles > 0) return true;
            if (!MANY) break;
        }
        return false;
    }
    // The next tile, of the next item after the last; false when there is none.
    __device__ __forceinline__ bool next(const AttnArgs &a, int q_tiles, int items) {
        step();
        if (++j < tiles) return true;
        if (!MANY) return false;
        j = 0;
        ++count;
        index += gridDim.x;
        return seek(a, q_tiles, items);
    }
    __device__ __forceinline__ void step() {
        ++tile;
        if (++stage == NS) {
            stage = 0;
            parity ^= 1;
        }
    }
    // Stage of the tile `back` < NS + 1 tiles ago, and its barriers' parity.
    __device__ __forceinline__ int stage_of(int back, int &its_parity) const {
        const int s = stage - back;
        its_parity = s < 0 ? parity ^ 1 : parity;
        return s < 0 ? s + NS : s;
    }
    __device__ __forceinline__ bool last() const { return j + 1 == tiles; }
    __device__ __forceinline__ bool tail() const { return last() && keys % kTcN != 0; }
};

template <typename T, int DP, int BIAS, int MODE>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_tc_fwd_kernel(const __grid_constant__ TcFwdArgs p) {
    using Sh = TcFwdShape<DP, MODE>;
    constexpr bool MANY = MODE == kFwdMany, SPLIT = MODE == kFwdSplit;
    constexpr int NS = Sh::kStages, NI = Sh::kItems;
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t q_full[NI], q_free[NI], o_free[NI], k_full[NS], v_full[NS], pv_done[NS],
        s_full[2], p_ready[2], landed, drained;
    __shared__ uint32_t tmem_base;
    __shared__ __align__(16) int s_rel[8][kTcHalf];
    __shared__ float s_top[2][2][kTcM];   // of the two threads of a query, in turn
    // at the end, with SPLIT: reference and the two halves of the sum
    float *s_m = s_top[0][0], *s_l = s_top[1][0];

    const AttnArgs &a = p.a;
    unsigned char *tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sQ = tiles, *sK = tiles + NI * Sh::kQBytes, *sV = sK + NS * Sh::kTileBytes;
    float *sBias = reinterpret_cast<float *>(tiles + Sh::kTileSmem);   // a window per stage
    const int q_tiles = (a.Lq + kTcM - 1) / kTcM, items = q_tiles * a.H * a.N;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (warp == kTcMmaWarp) {
        if (lane == 0) {
            for (int b = 0; b < NI; ++b) {
                mbar_init(&q_full[b], 1);
                mbar_init(&q_free[b], 1);
                mbar_init(&o_free[b], kTcSoft);
            }
            for (int s = 0; s < NS; ++s) {
                mbar_init(&k_full[s], 1);
                mbar_init(&v_full[s], 1);
                mbar_init(&pv_done[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[b], 2);   // the MMA thread, which saw the copies land, and its MMAs
                mbar_init(&p_ready[b], kTcSoft);
            }
            mbar_init(&landed, 1);
            mbar_init(&drained, 1);
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&tmem_base, Sh::kTmemCols);
        tcgen05_fence_before_sync();
    }
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = tmem_base;
    const float *bias0 = p.bias.base;
    wait_for_previous_kernel(bias0);
    bool ok = true;
    TcItem<NS, MODE> w = {};
    w.index = SPLIT ? blockIdx.x / cluster_size() : blockIdx.x;

    if (warp == kTcCopyWarp) {
        // ---------------------------------------------------- copies
        const float *bias = nullptr;
        int rq0 = 0, tails = 0;
        for (bool more = w.seek(a, q_tiles, items); more; more = w.next(a, q_tiles, items)) {
            const int s = w.stage;
            if (lane == 0) {
                if (w.j == 0) {
                    const int b = w.count % NI;
                    if (w.count >= NI) ok = tc_wait(&q_free[b], (w.count / NI - 1) & 1, a.err);
                    if (ok) {
                        mbar_arrive_expect_tx(&q_full[b], Sh::kQBytes);
                        tc_load<DP, kTcM>(sQ + b * Sh::kQBytes, p.q, w.n, w.h, w.i0, &q_full[b]);
                    }
                    if (BIAS) {
                        bias = bias0 + (int64_t)w.h * p.bias.stride;
                        rq0 = rel_q(a, w.i0);
                    }
                }
                if (ok && w.tile >= NS) ok = tc_wait(&pv_done[s], w.parity ^ 1, a.err);   // consumed
                if (ok) {
                    mbar_arrive_expect_tx(&k_full[s], Sh::kTileBytes + (BIAS == kBiasWindow ? p.bias.count * 4 : 0));
                    tc_load<DP, kTcN>(sK + s * Sh::kTileBytes, p.k, w.n, w.h, w.key0 + w.j * kTcN,
                                      &k_full[s]);
                    if (BIAS == kBiasWindow)
                        bulk_copy_g2s(sBias + s * p.bias.count,
                                      bias + bias_start(p.bias, rq0 - rel_k(a, w.key0 + w.j * kTcN)),
                                      p.bias.count * 4, &k_full[s]);
                    // a tile with masked keys is cleared before it counts as loaded
                    uint64_t *bar = w.tail() ? &landed : &v_full[s];
                    mbar_arrive_expect_tx(bar, Sh::kTileBytes);
                    tc_load<DP, kTcN>(sV + s * Sh::kTileBytes, p.v, w.n, w.h, w.key0 + w.j * kTcN, bar);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (w.tail()) {   // values of masked keys must not reach the product
                ok = __all_sync(0xffffffffu, tc_wait(&landed, tails++ & 1, a.err));
                if (!ok) break;
                tc_clear_rows<DP, kTcN>(sV + s * Sh::kTileBytes, w.keys - w.j * kTcN);
                if (lane == 0) mbar_arrive(&v_full[s]);
            }
        }
        // every copy lands before the block may leave (they have, unless a wait gave up)
        for (int t = max(0, w.tile - NS); t < w.tile; ++t) {
            tc_wait(&k_full[t % NS], (t / NS) & 1, a.err);
            tc_wait(&v_full[t % NS], (t / NS) & 1, a.err);
        }
        if (!ok && w.count > 0) tc_wait(&q_full[(w.count - 1) % NI], ((w.count - 1) / NI) & 1, a.err);
    } else if (warp == kTcMmaWarp) {
        // ---------------------------------------------------- MMAs, one thread
        if (lane == 0) {
            const uint32_t idesc_s = umma_idesc_f16(kBf16, kTcM, kTcN);
            const int steps = (a.D + 15) / 16;
            const uint32_t idesc_o = umma_idesc_f16_bmn(kBf16, kTcM, steps * 16);
            const uint32_t q_lo = umma_lo_kmajor(smem_u32(sQ)), k_lo = umma_lo_kmajor(smem_u32(sK));
            const uint32_t v_lo = umma_lo_mnmajor(smem_u32(sV), kTcN * 128);
            TcItem<NS, MODE> c = w;   // one tile ahead: its scores are issued before w's product
            bool c_more = c.seek(a, q_tiles, items), w_more = w.seek(a, q_tiles, items);
            const auto scores = [&] {
                const int s = c.stage, b = c.count % NI;
                if (c.j == 0) ok = tc_wait(&q_full[b], (c.count / NI) & 1, a.err);
                if (ok && c.tile >= 2) {   // the weights of two tiles ago are consumed
                    int parity;
                    const int s2 = c.stage_of(2, parity);
                    ok = tc_wait(&pv_done[s2], parity, a.err);
                }
                ok = ok && tc_wait(&k_full[s], c.parity, a.err);
                if (!ok) return;
                tcgen05_fence_after_sync();
                tc_scores<DP>(tmem + (c.tile & 1) * kTcN, q_lo + b * (Sh::kQBytes / 16),
                              k_lo + s * (Sh::kTileBytes / 16), idesc_s, steps);
                mbar_arrive(&s_full[c.tile & 1]);
                umma_commit(&s_full[c.tile & 1]);
                if (c.last()) umma_commit(&q_free[b]);
                c_more = c.next(a, q_tiles, items);
            };
            if (c_more) scores();
            while (w_more && ok) {
                if (c_more) scores();
                const int s = w.stage, b = w.count % NI;
                ok = ok && tc_wait(&v_full[s], w.parity, a.err);
                if (w.j == 0 && w.count >= NI)   // the output that was there is stored
                    ok = ok && tc_wait(&o_free[b], (w.count / NI - 1) & 1, a.err);
                ok = ok && tc_wait(&p_ready[w.tile & 1], (w.tile / 2) & 1, a.err);
                if (!ok) break;
                tcgen05_fence_after_sync();
                tc_weighted(tmem + Sh::kTmemO + b * DP, tmem + (w.tile & 1) * kTcN,
                            v_lo + s * (Sh::kTileBytes / 16), idesc_o, w.j > 0);
                umma_commit(&pv_done[s]);
                w_more = w.next(a, q_tiles, items);
            }
            if (!ok) {   // a wait gave up: let the MMAs end before TMEM is released
                umma_commit(&drained);
                tc_wait(&drained, 0, a.err);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- softmax
        // After a wait that gave up a thread goes on without waiting (and its warp
        // without storing), so that its partner finds it at every pair_sync.
        const auto wait = [&](uint64_t *bar, int parity) {
            if (ok) ok = tc_wait(bar, parity, a.err);
            __syncwarp();
        };
        const int pair = warp % 4, part = warp / 4, lane_row = pair * 32 + lane;
        const uint32_t my_tmem = (uint32_t)(pair * 32) << 16;   // this warp's TMEM lanes
        const int first = part * kTcHalf;                       // this thread's columns of a tile
        const float c2 = a.scale * kLog2e;
        const int inverse = 65536 / a.Wk + 1;
        int turn = 0;

        // Stores the output of a finished item: rows of `o_at` in TMEM times 1 / l.
        const auto store = [&](int n, int h, int i, uint32_t o_at, bool any, float m, float l) {
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            T *out = (T *)p.O + (((int64_t)n * a.Lq + i) * a.H + h) * a.D;
#pragma unroll 1
            for (int d = part * 32; d < a.D; d += 64) {
                uint32_t o[32];
                if (any) {
                    tmem_ld_x32(o_at + d, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
                if (i < a.Lq) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        if (d + k < a.D) {   // D is a multiple of 8
                            uint4 v;
                            uint32_t *u = &v.x;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                u[e] = pack2<T>(__uint_as_float(o[k + 2 * e]) * inv,
                                                __uint_as_float(o[k + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4 *>(out + d + k) = v;
                        }
                }
            }
            if (part == 0 && i < a.Lq && p.lse)
                p.lse[((int64_t)n * a.H + h) * a.Lq + i] = lse_of(m - kWeightShift<T>, l);
        };
        // The item before the current one, whose product ends while the first tile
        // of the current one is worked on.
        struct {
            int n, h, i, stage, parity, count;
            float m, l;
        } past = {};
        const auto finish = [&] {
            s_top[turn][part][lane_row] = past.l;   // the row's other half of the sum
            pair_sync(pair);
            const float l = past.l + s_top[turn][part ^ 1][lane_row];
            turn ^= 1;
            wait(&pv_done[past.stage], past.parity);
            const int b = past.count % NI;
            if (__all_sync(0xffffffffu, ok)) {
                tcgen05_fence_after_sync();
                store(past.n, past.h, past.i, tmem + Sh::kTmemO + b * DP + my_tmem, true, past.m, l);
                tcgen05_fence_before_sync();
            }
            mbar_arrive(&o_free[b]);
        };

        for (; w.index < items; w.index += gridDim.x) {
            w.decode(a, q_tiles);
            const int i = w.i0 + lane_row;
            if (w.tiles == 0) {   // no key: nothing comes from the other warps
                if (SPLIT) break;
                if (__all_sync(0xffffffffu, ok)) store(w.n, w.h, i, 0, false, 0.0f, 0.0f);
                if (!MANY) break;
                continue;
            }
            const float *bias = BIAS ? bias0 + (int64_t)w.h * p.bias.stride : nullptr;
            const int rq0 = BIAS ? rel_q(a, w.i0) : 0, rq = BIAS ? rel_q(a, min(i, a.Lq - 1)) : 0;
            const uint32_t to = tmem + Sh::kTmemO + w.count % NI * DP + my_tmem;
            TileWalk walk;
            if (BIAS) walk.init(a.Hk, a.Wk, a.P, w.key0);
            // the bias of this query and the next tile's first key, and where the
            // thread's columns start in the keys' grid
            const float *row = nullptr;
            int x = 0, rel = 0;
            const auto aim = [&] {
                if (BIAS == kBiasWindow)
                    row = sBias + w.stage * p.bias.count +
                          (rq - walk.rel - bias_start(p.bias, rq0 - walk.rel));
                else if (BIAS)
                    row = bias + rq - walk.rel;
                if (BIAS) walk.half(part, x, rel);
            };
            aim();
            float m = -INFINITY, l = 0.0f;
            for (w.j = 0; w.j < w.tiles; ++w.j) {
                const int live = w.keys - w.j * kTcN, buffer = w.tile & 1, phase = (w.tile >> 1) & 1;
                uint32_t r[kTcHalf];
                float b[kTcHalf];
                wait(&s_full[buffer], phase);
                tcgen05_fence_after_sync();
                const uint32_t ts = tmem + my_tmem + buffer * kTcN + first;
                tmem_start_ld_x32(ts, r);
                if (!BIAS) {
#pragma unroll
                    for (int c = 0; c < kTcHalf; ++c) b[c] = 0.0f;
                } else if (BIAS == kBiasWindow && p.bias.runs) {
                    bias_by_runs<-1>(row, x, rel, walk, b);
                } else {
                    bias_offsets(s_rel[warp], walk, first, live, inverse);
                    bias_by_table<-1>(row, s_rel[warp], b);
                }
                tmem_wait_ld(r);
                scale_and_bias(r, c2, b);
                if (live < kTcN) {   // masked keys, whatever they hold
                    asm volatile("" ::: "memory");   // a branch: the selects would cost every tile
#pragma unroll
                    for (int c = 0; c < kTcHalf; ++c)
                        if (first + c >= live) r[c] = __float_as_uint(-INFINITY);
                }
                float top4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTcHalf; c += 2)
                    top4[c / 2 % 4] =
                        max3(top4[c / 2 % 4], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                // a new reference for the pair's rows (also out of m = -inf): rare after
                // the first tile
                if (pair_any(pair, top > m + kLazyGrowth)) {
                    s_top[turn][part][lane_row] = top;
                    pair_sync(pair);
                    top = fmaxf(top, s_top[turn][part ^ 1][lane_row]);
                    turn ^= 1;
                    if (w.j > 0) {
                        const float keep = top == -INFINITY ? 1.0f : exp2_approx(m - top);
                        int parity;
                        const int s1 = w.stage_of(1, parity);
                        wait(&pv_done[s1], parity);
                        tcgen05_fence_after_sync();
#pragma unroll 1
                        for (int d = part * 32; d < DP; d += 64) {   // every other chunk of O
                            uint32_t o[32];
                            tmem_ld_x32(to + d, o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                            tmem_st_x32(to + d, o);
                        }
                        tmem_wait_st();
                        l *= keep;
                    }
                    m = top;
                }
                // the next tile's place, among the exponentials
                if (BIAS) walk.next();
                w.step();
                aim();
                // a row with no key yet: weights 0
                const float ref = m == -INFINITY ? 0.0f : m - kWeightShift<T>;
                float2 sum[2] = {};
                const float2 one = make_float2(1.0f, 1.0f), shift = make_float2(-ref, -ref);
                uint32_t u[kTcHalf / 2];
#pragma unroll
                for (int c = 0; c < kTcHalf; c += 2) {
                    float2 e = fma_f32x2(
                        make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), one, shift);
                    e.x = exp2_approx(e.x);
                    e.y = exp2_approx(e.y);
                    sum[c / 2 % 2] = fma_f32x2(e, one, sum[c / 2 % 2]);
                    u[c / 2] = pack2<T>(e.x, e.y);
                }
                tmem_st_x16(ts, u);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                tcgen05_fence_before_sync();
                mbar_arrive(&p_ready[buffer]);
                if (MANY && w.j == 0 && w.count > 0) finish();
            }
            past.n = w.n;
            past.h = w.h;
            past.i = i;
            past.stage = w.stage_of(1, past.parity);
            past.count = w.count++;
            past.m = m;
            past.l = l;
            if (!MANY) break;
        }
        if (SPLIT) {
            if (w.count > 0)   // after that nothing reads the tiles any more
                wait(&pv_done[past.stage], past.parity);
            const bool any = __all_sync(0xffffffffu, ok) && w.count > 0;
            pair_sync(pair);   // the other warp has read s_top
            if (part == 0) s_m[lane_row] = any ? past.m : -INFINITY;
            s_l[part * kTcM + lane_row] = any ? past.l : 0.0f;
            if (any) {
                tcgen05_fence_after_sync();
                float *mine = reinterpret_cast<float *>(tiles) + lane_row * Sh::kSharePitch;
#pragma unroll 1
                for (int d = part * 32; d < a.D; d += 64) {
                    uint32_t o[32];
                    tmem_ld_x32(tmem + Sh::kTmemO + my_tmem + d, o);
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *reinterpret_cast<uint4 *>(mine + d + k) =
                            make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                }
            }
        } else if (w.count > 0) {
            finish();
        }
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == kTcMmaWarp) tmem_dealloc(tmem, Sh::kTmemCols);
    if constexpr (SPLIT) {
        // join: each block takes its part of the rows, the blocks' shares in order
        const auto cluster = cooperative_groups::this_cluster();
        cluster.sync();
        const int ranks = cluster_size(), rows = kTcM / ranks, runs = a.D / 8;
        w.decode(a, q_tiles);
        for (int k = threadIdx.x; k < rows * runs; k += kTcThreads) {
            const int row = cluster_rank() * rows + k / runs, d = k % runs * 8, i = w.i0 + row;
            if (i >= a.Lq) break;   // and so are the rows of later k
            float m = -INFINITY, l = 0.0f, o[8] = {};
            for (int r = 0; r < ranks; ++r) m = fmaxf(m, *cluster.map_shared_rank(&s_m[row], r));
            for (int r = 0; r < ranks; ++r) {
                const float its = *cluster.map_shared_rank(&s_m[row], r);
                const float lr = *cluster.map_shared_rank(&s_l[row], r) +
                                 *cluster.map_shared_rank(&s_l[kTcM + row], r);
                if (its == -INFINITY && lr == 0.0f) continue;   // no key: its output may be anything
                const float f = exp2_approx(its - m);
                const float4 *from = reinterpret_cast<const float4 *>(cluster.map_shared_rank(
                    reinterpret_cast<float *>(tiles) + row * Sh::kSharePitch + d, r));
                const float4 u = from[0], v = from[1];
                const float x[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = fmaf(x[e], f, o[e]);
                l = fmaf(lr, f, l);
            }
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            uint4 v;
            uint32_t *u = &v.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = pack2<T>(o[2 * e] * inv, o[2 * e + 1] * inv);
            *reinterpret_cast<uint4 *>((T *)p.O + (((int64_t)w.n * a.Lq + i) * a.H + w.h) * a.D + d) = v;
            if (d == 0 && p.lse)
                p.lse[((int64_t)w.n * a.H + w.h) * a.Lq + i] = lse_of(m - kWeightShift<T>, l);
        }
        cluster.sync();   // shared memory stays until the others have read it
    }
}

template <typename T, int DP, int BIAS, int MODE>
cudaError_t launch_attn_tc_fwd_as(const TcFwdArgs &p, int64_t blocks, int cluster, cudaStream_t s) {
    using Sh = TcFwdShape<DP, MODE>;
    auto kernel = attn_tc_fwd_kernel<T, DP, BIAS, MODE>;
    static DeviceFlags ready;
    const cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kTcSmemOne);
    });
    if (e != cudaSuccess) return e;
    const int window = BIAS == kBiasWindow ? Sh::kStages * p.bias.count * 4 : 0;
    return launch_next(LaunchAs(BIAS != kBiasNone, cluster), kernel, (unsigned)blocks, kTcThreads,
                       Sh::kSmem + window, s, p);
}

// kFwdMany pays off where an item is so short that setting up a block for it
// weighs (8 x 8 windows, 4096 items of one key tile: 44.7 us, 59.6 with a block
// each); keeping count of the items costs a fifth of a long one (64 x 64 tokens,
// 2048 items of 64 tiles: 557 us and 466).
// kFwdSplit where items leave SMs free: as many blocks for one as the SMs hold at
// two each, of two key tiles at least (16 queries, 8 heads, 32768 keys, D 64: 45
// us, 277 with a block each; 3000 tokens, 2 heads, D 128: 30 and 49).
constexpr int kTcManyTiles = 4, kTcMaxSplit = 8;
template <typename T, int DP, int BIAS>
cudaError_t launch_attn_tc_fwd_by_length(const TcFwdArgs &p, cudaStream_t s) {
    const int64_t items = (int64_t)((p.a.Lq + kTcM - 1) / kTcM) * p.a.H * p.a.N;
    const int tiles = (p.a.Lk + kTcN - 1) / kTcN;
    int split = 1;
    while (split < kTcMaxSplit && items * split * 2 <= 2 * kTcSms && tiles >= split * 4) split *= 2;
    if (split > 1) return launch_attn_tc_fwd_as<T, DP, BIAS, kFwdSplit>(p, items * split, split, s);
    return items > 2 * kTcSms && tiles <= kTcManyTiles
               ? launch_attn_tc_fwd_as<T, DP, BIAS, kFwdMany>(p, 2 * kTcSms, 1, s)
               : launch_attn_tc_fwd_as<T, DP, BIAS, kFwdOne>(p, items, 1, s);
}

// Runs the tensor-core forward pass when it takes the pointers and strides;
// *used reports whether it did.
template <typename T>
cudaError_t launch_attn_tc_fwd(const AttnArgs &a, const AttnPtrs &ptr, const float *bias,
                               cudaStream_t s, bool *used) {
    *used = false;
    TcFwdArgs p;
    if (a.D % 8 != 0 || ((uintptr_t)ptr.O & 15u) || a.Lk == 0) return cudaSuccess;
    constexpr bool bf16 = __is_same(T, __nv_bfloat16);
    if (!tc_view(&p.q, ptr.Q, bf16, a.N, a.Lq, a.H, a.D, a.qs, kTcM) ||
        !tc_view(&p.k, ptr.K, bf16, a.N, a.Lk, a.H, a.D, a.ks, kTcN) ||
        !tc_view(&p.v, ptr.V, bf16, a.N, a.Lk, a.H, a.D, a.vs, kTcN))
        return cudaSuccess;
    *used = true;
    p.a = a;
    p.bias = tc_bias_of(a, false);
    p.bias.base = bias;
    p.bias.stride = a.bias_stride;
    p.O = ptr.O;
    p.lse = ptr.lse;
    const int mode = !bias ? kBiasNone : p.bias.count ? kBiasWindow : kBiasGlobal;
    const auto run = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        return mode == kBiasNone     ? launch_attn_tc_fwd_by_length<T, DP, kBiasNone>(p, s)
               : mode == kBiasWindow ? launch_attn_tc_fwd_by_length<T, DP, kBiasWindow>(p, s)
                                     : launch_attn_tc_fwd_by_length<T, DP, kBiasGlobal>(p, s);
    };
    return a.D <= 64 ? run(std::integral_constant<int, 64>()) : run(std::integral_constant<int, 128>());
}

}  // namespace gs
