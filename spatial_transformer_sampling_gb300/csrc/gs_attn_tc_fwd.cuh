// gs_attn_tc_fwd.cuh -- attention forward on the tensor cores (fp16 / bf16).
//
// One CTA per 128 queries of one head; it walks the keys 64 at a time:
//   S = Q K^T             tcgen05.mma, fp32 in TMEM, two buffers
//   p = 2^(c S + bias - m)  two softmax threads per query, m its running reference
//   O += p V              tcgen05.mma with p (16-bit) read from TMEM, where it
//                         overwrites the scores it came from
// so scores and weights never leave the SM.  The two threads of a query take 32
// keys each and exchange their maxima through shared memory.  One thread of a
// ninth warp issues the MMAs (the scores of tile j + 1 are computed while the
// softmax warps work on tile j), one of a tenth the TMA loads: issued by one
// warp with votes between, both took longer than the softmax.
//
// The reference m follows the row's maximum lazily: O and the row sum are
// rescaled only when the maximum has grown by more than 2^8 since (the final
// division cancels m; weights stay below 2^8, inside both 16-bit types).  The
// row sum is kept in fp32 from the unrounded weights.
//
// The bias of a tile comes to shared memory with the keys (TcBias).
#pragma once

#include "gs_attn_tc.cuh"

namespace gs {

struct TcFwdArgs {
    AttnArgs a;
    TcView q, k, v;
    TcBias bias;
    void *O;
    float *lse;
};

constexpr float kLazyGrowth = 8.0f;   // log2 of how far the maximum may outgrow the reference

// log2 of the weight at the reference: fp16 weights are kept 2^6 up, so that
// small ones stay clear of the type's subnormal range (2^14 at most).
template <typename T> constexpr float kWeightShift = 0.0f;
template <> constexpr float kWeightShift<__half> = 6.0f;

template <int DP> struct TcFwdShape {
    static constexpr int kStages = DP == 64 ? 3 : 2;
    static constexpr int kQBytes = kTcM * DP * 2;
    static constexpr int kTileBytes = kTcN * DP * 2;
    static constexpr int kTileSmem = kQBytes + 2 * kStages * kTileBytes;
    static constexpr int kSmem = kTileSmem + 1024;   // 1024-byte alignment of the tiles
    static constexpr int kTmemCols = 256;            // two score buffers, O; two CTAs per SM
    static constexpr int kTmemO = 2 * kTcN;
};

template <typename T, int DP, int BIAS>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_tc_fwd_kernel(const __grid_constant__ TcFwdArgs p) {
    using Sh = TcFwdShape<DP>;
    constexpr int NS = Sh::kStages;
    constexpr bool kBf16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t q_full, k_full[NS], v_full[NS], s_full[2], p_ready[2], pv_done[NS], cleared;
    __shared__ uint32_t tmem_base;

    const AttnArgs &a = p.a;
    unsigned char *tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sQ = tiles, *sK = tiles + Sh::kQBytes, *sV = sK + NS * Sh::kTileBytes;
    float *sBias = reinterpret_cast<float *>(tiles + Sh::kTileSmem);   // a window per stage
    __shared__ __align__(16) int s_rel[8][kTcHalf];
    __shared__ float s_top[2][2][kTcM];   // of the two threads of a query, in turn

    const int q_tiles = (a.Lq + kTcM - 1) / kTcM;
    const int i0 = (int)(blockIdx.x % q_tiles) * kTcM;
    const int h = (int)(blockIdx.x / q_tiles % a.H), n = (int)(blockIdx.x / q_tiles / a.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // entry of relative index 0, and the first query's index
    const float *bias = BIAS ? p.bias.base + (int64_t)h * p.bias.stride : nullptr;
    const int rq0 = rel_q(a, i0);
    const int keys = keys_of(a, n), T_tiles = (keys + kTcN - 1) / kTcN;

    if (warp == kTcMmaWarp) {
        if (lane == 0) {
            mbar_init(&q_full, 1);
            for (int s = 0; s < NS; ++s) {
                mbar_init(&k_full[s], 1);
                mbar_init(&v_full[s], 1);
                mbar_init(&pv_done[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[b], 2);   // the MMA thread, which saw the copies land, and its MMAs
                mbar_init(&p_ready[b], kTcSoft);
            }
            mbar_init(&cleared, 1);
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&tmem_base, Sh::kTmemCols);
        tcgen05_fence_before_sync();
    }
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = tmem_base, tmem_o = tmem + Sh::kTmemO;
    bool ok = true;

    const bool tail = keys % kTcN != 0;   // the last tile holds masked keys

    if (warp == kTcCopyWarp) {
        // ---------------------------------------------------- copies
        if (lane == 0 && T_tiles > 0) {
            mbar_arrive_expect_tx(&q_full, Sh::kQBytes);
            tc_load<DP, kTcM>(sQ, p.q, n, h, i0, &q_full);
            for (int t = 0; t < T_tiles; ++t) {
                const int s = t % NS;
                if (t >= NS) {   // the stage's last tile is consumed
                    ok = tc_wait(&pv_done[s], (t / NS - 1) & 1, a.err);
                    if (!ok) break;
                }
                mbar_arrive_expect_tx(&k_full[s], Sh::kTileBytes + (BIAS == kBiasWindow ? p.bias.count * 4 : 0));
                tc_load<DP, kTcN>(sK + s * Sh::kTileBytes, p.k, n, h, t * kTcN, &k_full[s]);
                if (BIAS == kBiasWindow)
                    bulk_copy_g2s(sBias + s * p.bias.count,
                                  bias + bias_start(p.bias, rq0 - rel_k(a, t * kTcN)),
                                  p.bias.count * 4, &k_full[s]);
                mbar_arrive_expect_tx(&v_full[s], Sh::kTileBytes);
                tc_load<DP, kTcN>(sV + s * Sh::kTileBytes, p.v, n, h, t * kTcN, &v_full[s]);
            }
        }
        __syncwarp();
        if (T_tiles > 0 && tail) {   // values of masked keys must not reach the product
            const int t = T_tiles - 1;
            ok = tc_wait(&v_full[t % NS], (t / NS) & 1, a.err);
            __syncwarp();
            tc_clear_rows<DP, kTcN>(sV + t % NS * Sh::kTileBytes, keys - t * kTcN);
            if (lane == 0) mbar_arrive(&cleared);
        }
        // every copy lands before the block may leave (they have, unless a wait gave up)
        for (int t = max(0, T_tiles - NS); t < T_tiles; ++t) {
            tc_wait(&k_full[t % NS], (t / NS) & 1, a.err);
            tc_wait(&v_full[t % NS], (t / NS) & 1, a.err);
        }
    } else if (warp == kTcMmaWarp) {
        // ---------------------------------------------------- MMAs, one thread
        if (lane == 0 && T_tiles > 0) {
            const uint32_t idesc_s = umma_idesc_f16(kBf16, kTcM, kTcN);
            const int steps = (a.D + 15) / 16;
            const uint32_t idesc_o = umma_idesc_f16_bmn(kBf16, kTcM, steps * 16);
            const uint32_t q_lo = umma_lo_kmajor(smem_u32(sQ)), k_lo = umma_lo_kmajor(smem_u32(sK));
            const uint32_t v_lo = umma_lo_mnmajor(smem_u32(sV), kTcN * 128);
            ok = tc_wait(&q_full, 0, a.err) && tc_wait(&k_full[0], 0, a.err);
            if (ok) {
                tc_scores<DP>(tmem, q_lo, k_lo, idesc_s, steps);
                mbar_arrive(&s_full[0]);
                umma_commit(&s_full[0]);
            }
            for (int j = 0; j < T_tiles && ok; ++j) {
                const int s = j % NS;
                if (j + 1 < T_tiles) {   // scores into the other buffer: its weights are consumed
                    const int s1 = (j + 1) % NS;
                    if (j > 0) ok = tc_wait(&pv_done[(j - 1) % NS], ((j - 1) / NS) & 1, a.err);
                    ok = ok && tc_wait(&k_full[s1], ((j + 1) / NS) & 1, a.err);
                    if (!ok) break;
                    tcgen05_fence_after_sync();
                    tc_scores<DP>(tmem + ((j + 1) & 1) * kTcN, q_lo, k_lo + s1 * (Sh::kTileBytes / 16),
                                  idesc_s, steps);
                    mbar_arrive(&s_full[(j + 1) & 1]);
                    umma_commit(&s_full[(j + 1) & 1]);
                }
                ok = tc_wait(&v_full[s], (j / NS) & 1, a.err);
                if (tail && j == T_tiles - 1) ok = ok && tc_wait(&cleared, 0, a.err);
                ok = ok && tc_wait(&p_ready[j & 1], (j / 2) & 1, a.err);
                if (!ok) break;
                tcgen05_fence_after_sync();
                tc_weighted(tmem_o, tmem + (j & 1) * kTcN, v_lo + s * (Sh::kTileBytes / 16), idesc_o,
                            j > 0);
                umma_commit(&pv_done[s]);
            }
            if (!ok) {   // a wait gave up: let the MMAs end before TMEM is released
                umma_commit(&q_full);
                tc_wait(&q_full, 1, a.err);
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
        const int i = i0 + lane_row;
        const float c2 = a.scale * kLog2e;
        const int rq = BIAS ? rel_q(a, min(i, a.Lq - 1)) : 0;
        TileWalk walk;
        if (BIAS) walk.init(a.Hk, a.Wk, a.P);
        const int inverse = 65536 / a.Wk + 1;
        float m = -INFINITY, l = 0.0f;
        int stage = 0, turn = 0;
        // the bias of this query and the next tile's first key, and where the
        // thread's columns start in the keys' grid
        const float *row = nullptr;
        int x = 0, rel = 0;
        const auto aim = [&] {
            if (BIAS == kBiasWindow)
                row = sBias + stage * p.bias.count +
                      (rq - walk.rel - bias_start(p.bias, rq0 - walk.rel));
            else if (BIAS)
                row = bias + rq - walk.rel;
            if (BIAS) walk.half(part, x, rel);
        };
        aim();
        for (int j = 0; j < T_tiles; ++j) {
            const int live = keys - j * kTcN;
            uint32_t r[kTcHalf];
            float b[kTcHalf];
            wait(&s_full[j & 1], (j / 2) & 1);
            tcgen05_fence_after_sync();
            const uint32_t ts = tmem + my_tmem + (j & 1) * kTcN + first;
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
                if (j > 0) {
                    const float keep = top == -INFINITY ? 1.0f : exp2_approx(m - top);
                    wait(&pv_done[(j - 1) % NS], ((j - 1) / NS) & 1);
                    tcgen05_fence_after_sync();
                    const uint32_t to = tmem_o + my_tmem;
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
            if (++stage == NS) stage = 0;
            aim();
            // a row with no key yet: weights 0
            const float ref = m == -INFINITY ? 0.0f : m - kWeightShift<T>;
            float2 sum[2] = {};
            const float2 one = make_float2(1.0f, 1.0f), shift = make_float2(-ref, -ref);
            uint32_t w[kTcHalf / 2];
#pragma unroll
            for (int c = 0; c < kTcHalf; c += 2) {
                float2 e = fma_f32x2(
                    make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), one, shift);
                e.x = exp2_approx(e.x);
                e.y = exp2_approx(e.y);
                sum[c / 2 % 2] = fma_f32x2(e, one, sum[c / 2 % 2]);
                w[c / 2] = pack2<T>(e.x, e.y);
            }
            tmem_st_x16(ts, w);
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tmem_wait_st();
            tcgen05_fence_before_sync();
            mbar_arrive(&p_ready[j & 1]);
        }
        // the product before the last may be unfinished here, but the one a stage
        // earlier is done, so the phase's parity tells
        if (T_tiles > 0) wait(&pv_done[(T_tiles - 1) % NS], ((T_tiles - 1) / NS) & 1);
        s_top[turn][part][lane_row] = l;   // the row's other half of the sum
        pair_sync(pair);
        l += s_top[turn][part ^ 1][lane_row];
        if (__all_sync(0xffffffffu, ok)) {
            tcgen05_fence_after_sync();
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            T *out = (T *)p.O + (((int64_t)n * a.Lq + i) * a.H + h) * a.D;
#pragma unroll 1
            for (int d = part * 32; d < a.D; d += 64) {
                uint32_t o[32];
                if (T_tiles > 0) {
                    tmem_ld_x32(tmem_o + my_tmem + d, o);
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
                if (i < a.Lq) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        if (d + k < a.D) {   // D is a multiple of 8
                            uint4 w;
                            uint32_t *u = &w.x;
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                u[e] = pack2<T>(__uint_as_float(o[k + 2 * e]) * inv,
                                                __uint_as_float(o[k + 2 * e + 1]) * inv);
                            *reinterpret_cast<uint4 *>(out + d + k) = w;
                        }
                }
            }
            if (part == 0 && i < a.Lq && p.lse)
                p.lse[((int64_t)n * a.H + h) * a.Lq + i] =
                    l != 0.0f ? (m - kWeightShift<T> + log2f(l)) * kLn2 : -INFINITY;
        }
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == kTcMmaWarp) tmem_dealloc(tmem, Sh::kTmemCols);
}

template <typename T, int DP, int BIAS>
cudaError_t launch_attn_tc_fwd_as(const TcFwdArgs &p, cudaStream_t s) {
    using Sh = TcFwdShape<DP>;
    auto kernel = attn_tc_fwd_kernel<T, DP, BIAS>;
    static DeviceFlags ready;
    const cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kTcSmemOne);
    });
    if (e != cudaSuccess) return e;
    const int window = BIAS == kBiasWindow ? Sh::kStages * p.bias.count * 4 : 0;
    const int64_t blocks = (int64_t)((p.a.Lq + kTcM - 1) / kTcM) * p.a.H * p.a.N;
    kernel<<<(unsigned)blocks, kTcThreads, Sh::kSmem + window, s>>>(p);
    return cudaGetLastError();
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
        return mode == kBiasNone     ? launch_attn_tc_fwd_as<T, DP, kBiasNone>(p, s)
               : mode == kBiasWindow ? launch_attn_tc_fwd_as<T, DP, kBiasWindow>(p, s)
                                     : launch_attn_tc_fwd_as<T, DP, kBiasGlobal>(p, s);
    };
    return a.D <= 64 ? run(std::integral_constant<int, 64>()) : run(std::integral_constant<int, 128>());
}

}  // namespace gs
