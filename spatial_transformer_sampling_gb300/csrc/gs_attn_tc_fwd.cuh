// gs_attn_tc_fwd.cuh -- attention forward on the tensor cores (fp16 / bf16).
//
// One CTA per 128 queries of one head; it walks the keys 64 at a time:
//   S = Q K^T             tcgen05.mma, fp32 in TMEM, two buffers
//   p = 2^(c S + bias - m)  one softmax thread per query, m its running reference
//   O += p V              tcgen05.mma with p (16-bit) read from TMEM, where it
//                         overwrites the scores it came from
// so scores and weights never leave the SM.  A fifth warp issues the TMA loads
// and the MMAs: the scores of tile j + 1 are computed while the softmax warps
// work on tile j.
//
// The reference m follows the row's maximum lazily: O and the row sum are
// rescaled only when the maximum has grown by more than 2^8 since (the final
// division cancels m; weights stay below 2^8, inside both 16-bit types).  The
// row sum is kept in fp32 from the unrounded weights.
//
// The bias of the CTA's rows is a window of the expanded bias, contiguous in
// the relative index: it is copied to shared memory once (`bias_window` floats)
// when it fits beside the tiles of two CTAs per SM, else read through L1.
#pragma once

#include "gs_attn_tc.cuh"

namespace gs {

struct TcFwdArgs {
    AttnArgs a;
    TcView q, k, v;
    const float *bias;   // expanded (H, R), or nullptr
    int bias_window;     // floats of shared memory for the bias (0: read global memory)
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

template <typename T, int DP, bool BIAS>
__global__ void __launch_bounds__(kTcThreads, 2)
    attn_tc_fwd_kernel(const __grid_constant__ TcFwdArgs p) {
    using Sh = TcFwdShape<DP>;
    constexpr int NS = Sh::kStages;
    constexpr bool kBf16 = sizeof(T) == 2 && __is_same(T, __nv_bfloat16);
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t q_full, k_full[NS], v_full[NS], s_full[2], p_ready[2], pv_done, drained;
    __shared__ uint32_t tmem_base;

    const AttnArgs &a = p.a;
    unsigned char *tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sQ = tiles, *sK = tiles + Sh::kQBytes, *sV = sK + NS * Sh::kTileBytes;
    float *sBias = reinterpret_cast<float *>(tiles + Sh::kTileSmem);

    const int q_tiles = (a.Lq + kTcM - 1) / kTcM;
    const int i0 = (int)(blockIdx.x % q_tiles) * kTcM;
    const int h = (int)(blockIdx.x / q_tiles % a.H), n = (int)(blockIdx.x / q_tiles / a.H);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int keys = keys_of(a, n), T_tiles = (keys + kTcN - 1) / kTcN;

    if (warp == 4) {
        if (lane == 0) {
            mbar_init(&q_full, 1);
            for (int s = 0; s < NS; ++s) {
                mbar_init(&k_full[s], 1);
                mbar_init(&v_full[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[b], 1);
                mbar_init(&p_ready[b], kTcM);
            }
            mbar_init(&pv_done, 1);
            mbar_init(&drained, 1);
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&tmem_base, Sh::kTmemCols);
        tcgen05_fence_before_sync();
    }
    // the window of relative indices that this CTA's pairs fall into
    const int i_last = min(i0 + kTcM, a.Lq) - 1;
    const float *bias = nullptr;
    int rel_base = 0;
    if (BIAS && keys > 0) {
        bias = p.bias + (int64_t)h * a.R;
        if (p.bias_window) {
            rel_base = rel_q(a, i0) - rel_k(a, keys - 1);
            const int count = rel_q(a, i_last) - rel_base + 1;
            for (int r = threadIdx.x; r < count; r += kTcThreads) sBias[r] = __ldg(bias + rel_base + r);
            bias = sBias;
        }
    }
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = tmem_base, tmem_o = tmem + Sh::kTmemO;
    bool ok = true;

    if (warp == 4) {
        // ---------------------------------------------------- copies and MMAs
        const uint32_t idesc_s = umma_idesc_f16(kBf16, kTcM, kTcN);
        const int width = (a.D + 15) / 16 * 16;
        const uint32_t idesc_o = umma_idesc_f16_bmn(kBf16, kTcM, width);
        const uint32_t q_at = smem_u32(sQ), k_at = smem_u32(sK), v_at = smem_u32(sV);
        const auto load = [&](int t) {   // one lane
            const int s = t % NS;
            mbar_arrive_expect_tx(&k_full[s], Sh::kTileBytes);
            tc_load<DP, kTcN>(sK + s * Sh::kTileBytes, p.k, n, h, t * kTcN, &k_full[s]);
            mbar_arrive_expect_tx(&v_full[s], Sh::kTileBytes);
            tc_load<DP, kTcN>(sV + s * Sh::kTileBytes, p.v, n, h, t * kTcN, &v_full[s]);
        };
        int loaded = 0;   // tiles whose copies were issued
        if (lane == 0 && T_tiles > 0) {
            mbar_arrive_expect_tx(&q_full, Sh::kQBytes);
            tc_load<DP, kTcM>(sQ, p.q, n, h, i0, &q_full);
            for (; loaded < NS && loaded < T_tiles; ++loaded) load(loaded);
        }
        loaded = __shfl_sync(0xffffffffu, loaded, 0);
        if (T_tiles > 0) {
            ok = mbar_wait_bounded(&q_full, 0, a.err) && mbar_wait_bounded(&k_full[0], 0, a.err);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) {
                tc_scores<kTcN>(tmem, q_at, k_at, idesc_s, width / 16);
                umma_commit(&s_full[0]);
            }
        }
        for (int j = 0; j < T_tiles && ok; ++j) {
            const int s = j % NS, ph = (j / NS) & 1;
            if (j > 0) {   // tile j - 1 is consumed: its stage takes the next copy
                ok = mbar_wait_bounded(&pv_done, (j - 1) & 1, a.err);
                if (__any_sync(0xffffffffu, !ok)) break;
                if (loaded < T_tiles) {
                    if (lane == 0) load(loaded);
                    ++loaded;
                }
            }
            if (j + 1 < T_tiles) {   // the other score buffer: its weights are consumed
                const int s1 = (j + 1) % NS;
                ok = mbar_wait_bounded(&k_full[s1], ((j + 1) / NS) & 1, a.err);
                if (__any_sync(0xffffffffu, !ok)) break;
                if (lane == 0) {
                    tcgen05_fence_after_sync();
                    tc_scores<kTcN>(tmem + ((j + 1) & 1) * kTcN, q_at, k_at + s1 * Sh::kTileBytes,
                                    idesc_s, width / 16);
                    umma_commit(&s_full[(j + 1) & 1]);
                }
            }
            ok = mbar_wait_bounded(&v_full[s], ph, a.err);
            if (__any_sync(0xffffffffu, !ok)) break;
            if (keys - j * kTcN < kTcN)
                tc_clear_rows<DP, kTcN>(sV + s * Sh::kTileBytes, keys - j * kTcN);
            ok = mbar_wait_bounded(&p_ready[j & 1], (j / 2) & 1, a.err);
            if (__any_sync(0xffffffffu, !ok)) break;
            if (lane == 0) {
                tcgen05_fence_after_sync();
                tc_weighted<kTcN>(tmem_o, tmem + (j & 1) * kTcN, v_at + s * Sh::kTileBytes, idesc_o,
                                  j > 0);
                umma_commit(&pv_done);
            }
        }
        if (!__all_sync(0xffffffffu, ok)) {
            // a wait gave up: let this CTA's copies and MMAs end before it leaves
            if (lane == 0) umma_commit(&drained);
            mbar_wait_bounded(&drained, 0, a.err);
            for (int t = max(0, loaded - NS); t < loaded; ++t) {
                mbar_wait_bounded(&k_full[t % NS], (t / NS) & 1, a.err);
                mbar_wait_bounded(&v_full[t % NS], (t / NS) & 1, a.err);
            }
        }
    } else {
        // ---------------------------------------------------- softmax, a row per thread
        const uint32_t my_tmem = (uint32_t)(warp * 32) << 16;   // this warp's TMEM lanes
        const int i = i0 + threadIdx.x;
        const float c2 = a.scale * kLog2e;
        const float *row = BIAS && keys > 0 ? bias + (rel_q(a, min(i, a.Lq - 1)) - rel_base) : nullptr;
        float m = -INFINITY, l = 0.0f;
        for (int j = 0; j < T_tiles; ++j) {
            const int live = keys - j * kTcN;
            uint32_t r[64];
            ok = mbar_wait_bounded(&s_full[j & 1], (j / 2) & 1, a.err);
            if (__any_sync(0xffffffffu, !ok)) break;
            tcgen05_fence_after_sync();
            const uint32_t ts = tmem + my_tmem + (j & 1) * kTcN;
            tmem_ld_x32<0>(ts, r);
            tmem_ld_x32<32>(ts + 32, r);
            tmem_wait_ld<0>(r);
            tmem_wait_ld<32>(r);
            if (BIAS) {
                const int y = j * kTcN / a.Wk, x = j * kTcN - y * a.Wk;
                for_each_bias<-1>(
                    row, x, y * a.P + x, a.Wk, a.P, live,
                    [&](int c, float b) {
                        r[c] = __float_as_uint(fmaf(__uint_as_float(r[c]), c2, b));
                    },
                    [&](int c) { r[c] = __float_as_uint(-INFINITY); });
            } else {
#pragma unroll
                for (int c = 0; c < kTcN; ++c)
                    r[c] = __float_as_uint(c < live ? __uint_as_float(r[c]) * c2 : -INFINITY);
            }
            float top = m;
#pragma unroll
            for (int c = 0; c < kTcN; ++c) top = fmaxf(top, __uint_as_float(r[c]));
            // (top > m + growth) also takes a row out of m = -inf
            if (j == 0) {
                m = top;
            } else if (__any_sync(0xffffffffu, top > m + kLazyGrowth)) {
                const float keep = top == -INFINITY ? 1.0f : exp2_approx(m - top);
                ok = mbar_wait_bounded(&pv_done, (j - 1) & 1, a.err);
                if (__any_sync(0xffffffffu, !ok)) break;
                tcgen05_fence_after_sync();
                const uint32_t to = tmem_o + my_tmem;
#pragma unroll 1
                for (int d = 0; d < DP; d += 32) {
                    uint32_t o[32];
                    tmem_ld_x32<0>(to + d, o);
                    tmem_wait_ld<0>(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                    tmem_st_x32(to + d, o);
                }
                tmem_wait_st();
                l *= keep;
                m = top;
            }
            // a row with no key yet: weights 0
            const float ref = m == -INFINITY ? 0.0f : m - kWeightShift<T>;
            float2 sum[4] = {};
            const float2 one = make_float2(1.0f, 1.0f), shift = make_float2(-ref, -ref);
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < kTcN; c += 2) {
                float2 e = fma_f32x2(
                    make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), one, shift);
                e.x = exp2_approx(e.x);
                e.y = exp2_approx(e.y);
                sum[c / 2 % 4] = fma_f32x2(e, one, sum[c / 2 % 4]);
                w[c / 2] = pack2<T>(e.x, e.y);
            }
            tmem_st_x32(ts, w);
            l += ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y)) +
                 ((sum[2].x + sum[2].y) + (sum[3].x + sum[3].y));
            tmem_wait_st();
            tcgen05_fence_before_sync();
            mbar_arrive(&p_ready[j & 1]);
        }
        // S of the last tile was ready before the product of the one before it
        // had to be, so this warp may be two phases ahead of pv_done: a parity
        // wait tells neighbouring phases apart only, hence both in turn
        if (__all_sync(0xffffffffu, ok) && T_tiles > 1)
            ok = mbar_wait_bounded(&pv_done, (T_tiles - 2) & 1, a.err);
        if (__all_sync(0xffffffffu, ok) && T_tiles > 0)
            ok = mbar_wait_bounded(&pv_done, (T_tiles - 1) & 1, a.err);
        if (__all_sync(0xffffffffu, ok)) {
            tcgen05_fence_after_sync();
            const float inv = l != 0.0f ? 1.0f / l : 0.0f;
            T *out = (T *)p.O + (((int64_t)n * a.Lq + i) * a.H + h) * a.D;
#pragma unroll 1
            for (int d = 0; d < a.D; d += 32) {
                uint32_t o[32];
                if (T_tiles > 0) {
                    tmem_ld_x32<0>(tmem_o + my_tmem + d, o);
                    tmem_wait_ld<0>(o);
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
            if (i < a.Lq && p.lse)
                p.lse[((int64_t)n * a.H + h) * a.Lq + i] =
                    l != 0.0f ? (m - kWeightShift<T> + log2f(l)) * kLn2 : -INFINITY;
        }
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == 4) tmem_dealloc(tmem, Sh::kTmemCols);
}

template <typename T, int DP, bool BIAS>
cudaError_t launch_attn_tc_fwd_as(TcFwdArgs &p, cudaStream_t s) {
    using Sh = TcFwdShape<DP>;
    auto kernel = attn_tc_fwd_kernel<T, DP, BIAS>;
    static DeviceFlags ready;
    cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kTcSmemTwo);
    });
    if (e != cudaSuccess) return e;
    const int64_t window = BIAS ? tc_bias_window(p.a, false) : 0;
    p.bias_window = Sh::kSmem + window * 4 <= kTcSmemTwo ? (int)window : 0;
    const int64_t blocks = (int64_t)((p.a.Lq + kTcM - 1) / kTcM) * p.a.H * p.a.N;
    kernel<<<(unsigned)blocks, kTcThreads, Sh::kSmem + p.bias_window * 4, s>>>(p);
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
    p.bias = bias;
    p.O = ptr.O;
    p.lse = ptr.lse;
    if (a.D <= 64)
        return bias ? launch_attn_tc_fwd_as<T, 64, true>(p, s) : launch_attn_tc_fwd_as<T, 64, false>(p, s);
    return bias ? launch_attn_tc_fwd_as<T, 128, true>(p, s) : launch_attn_tc_fwd_as<T, 128, false>(p, s);
}

}  // namespace gs
