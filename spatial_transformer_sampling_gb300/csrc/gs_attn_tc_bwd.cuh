// gs_attn_tc_bwd.cuh -- attention backward on the tensor cores (fp16 / bf16).
//
// Two kinds of blocks in one launch, so that every gradient is summed by one CTA in one
// order (no atomics):
//   DKV: 128 keys per CTA against the queries, 64 at a time;
//   DQ:  128 queries per CTA against the keys, 64 at a time.
// With rows R1, R2 (DKV: K, V; DQ: Q, dO) resident and columns C1, C2 (DKV:
// Q, dO; DQ: K, V) streamed by TMA, each step computes
//   S  = R1 C1^T,  dP = R2 C2^T             tcgen05.mma, fp32 in TMEM
//   p  = 2^(c S + bias - lse),  ds = p (dP - delta)   two threads per row
//   acc1 += ds C1  (dK or dQ),  acc2 += p C2  (dV)    tcgen05.mma
// p and ds are rounded to the 16-bit type (both operands of the matrix instruction
// have one; 2.4e-3 of a gradient in bf16 with the store's 1.7e-3) and read back from
// TMEM, where they overwrite dP; S is free as soon as it is loaded, so the next step's S is
// computed while the softmax warps work.  The scores are computed in both
// kinds (7 products instead of 5): the alternative, dQ summed across CTAs,
// needs fp32 atomics, whose order would change the result.
//
// Bound by the latency of the chain scores, weights, ds and (DQ) the bias
// gradient's window, which takes about as long as the softmax: half of the issue
// slots, 43 % of the shared-memory wavefronts, 17 % of the tensor pipe.  8 x 8
// heads of 32 x 32 tokens, D 64, bf16, ragged, with bias: 121 us.
#pragma once

#include "gs_attn_rel.cuh"
#include "gs_attn_tc.cuh"

namespace gs {

struct TcBwdArgs {
    AttnArgs a;
    TcView r1, r2, c1, c2;
    TcBias bias;
    const float *lse2;        // (N, H, rows64(Lq)): lse * log2(e), +inf where nothing counts
    const float *delta;       // same shape: dO . O
    RangeArgs range;          // fp16: what bounds ds
    void *out1, *out2;        // dK, dV or dQ
    RelArgs rel;              // DQ: the bias gradient
};

template <int DP, bool DKV> struct TcBwdShape {
    static constexpr int kStages = 2;
    static constexpr int kRowBytes = kTcM * DP * 2;
    static constexpr int kTileBytes = kTcN * DP * 2;
    static constexpr int kVecBytes = DKV ? 2 * kTcN * 4 : 0;   // lse2, delta of the columns
    static constexpr int kTileSmem = 2 * kRowBytes + 2 * kStages * kTileBytes;
    static constexpr int kSmem = kTileSmem + kStages * kVecBytes + 1024;
    static constexpr int kTmemS = 0, kTmemP = kTcN, kTmemAcc1 = 2 * kTcN, kTmemAcc2 = 2 * kTcN + DP;
    static constexpr int kTmemCols = DKV && DP == 128 ? 512 : 256;
    static constexpr int kCtas = kSmem <= 227 * 1024 / 2 - 1024 ? 2 : 1;
};

// Weights are at most 1: fp16 ones are scaled by 2^12 on their way to the
// tensor cores (and dV back), so that those below 2^-14 keep their precision.
template <typename T> constexpr float kWeightScale = 1.0f;
template <> constexpr float kWeightScale<__half> = 4096.0f;

// Their gradients ds go with dO, which may be anything between a mean's over all
// tokens and a scaled loss's: fp16 ones are multiplied by the power of two that
// takes the bound of a (batch, head) pair to 2^15 at most (dK and dQ are divided
// by it again).  Unscaled, a dO of 1e-4 over 4096 keys left ds below 2^-14, with 5 %
// of dK lost, and one of 2e4 over 64 keys took it beyond the type's range.
template <typename T> constexpr bool kScaledGradient = __is_same(T, __half);

// That power of two; a whole warp calls it.
__device__ __forceinline__ float gradient_scale(const float *most, int parts, int nh) {
    const int lane = threadIdx.x % 32;
    float g = 0.0f, v = 0.0f;
    if (lane < parts) {
        const float2 both = *reinterpret_cast<const float2 *>(most + ((int64_t)nh * parts + lane) * 2);
        g = both.x;
        v = both.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    }
    // |ds| <= 2 sqrt(g v) < 2^(1 + e / 2) with e the exponent above g v: both are sums
    // of 128 squares of fp16 values, 2^-48 to 2^39, so that the scale is 2^-26 to 2^62
    const float square = g * v;
    if (!(square > 0.0f)) return 1.0f;
    const int e = (int)(__float_as_uint(square) >> 23) - 126;
    return __uint_as_float((uint32_t)(127 + 14 - ((e + 1) >> 1)) << 23);
}

template <typename T, int DP, int BIAS, bool DKV>
__device__ __forceinline__ void attn_tc_bwd_block(const TcBwdArgs &p, int block) {
    using Sh = TcBwdShape<DP, DKV>;
    constexpr int NS = Sh::kStages;
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t r_full, c_full[NS], s_full, s_free, dp_full, pd_ready, done[NS], finished, cleared;
    __shared__ uint32_t tmem_base;

    const AttnArgs &a = p.a;
    unsigned char *tiles = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *sR1 = tiles, *sR2 = sR1 + Sh::kRowBytes, *sC1 = sR2 + Sh::kRowBytes,
                  *sC2 = sC1 + NS * Sh::kTileBytes;
    float *sVec = reinterpret_cast<float *>(tiles + Sh::kTileSmem);
    float *sRel = sVec + NS * Sh::kVecBytes / 4;
    float *sBias = sRel + rel_smem(p.rel.window, 4) / 4;   // a window per stage
    __shared__ __align__(16) int s_rel[8][kTcHalf];

    const int rows = DKV ? a.Lk : a.Lq;
    const int row_tiles = (rows + kTcM - 1) / kTcM;
    const int i0 = block % row_tiles * kTcM;
    const int nh = p.rel.head0 + block / row_tiles;
    const int h = nh % a.H, n = nh / a.H;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int keys = keys_of(a, n);
    const int live_rows = DKV ? keys : a.Lq;    // rows from here on get zeros
    const int cols = i0 < live_rows ? (DKV ? a.Lq : keys) : 0;
    const int steps = (cols + kTcN - 1) / kTcN;
    const float *lse2 = p.lse2 + (int64_t)nh * rows64(a.Lq);
    const float *delta = p.delta + (int64_t)nh * rows64(a.Lq);

    // entry of relative index 0, the first row's part of it, and the index at
    // which the first row meets column `col`
    const float *bias = BIAS ? p.bias.base + (int64_t)h * p.bias.stride : nullptr;
    const int row0 = DKV ? -rel_k(a, i0) : rel_q(a, i0);
    const auto meet = [&](int col) { return row0 + (DKV ? rel_q(a, col) : -rel_k(a, col)); };

    if (warp == kTcMmaWarp) {
        if (lane == 0) {
            mbar_init(&r_full, 1);
            for (int s = 0; s < NS; ++s) {
                mbar_init(&c_full[s], 1);
                mbar_init(&done[s], 1);
            }
            mbar_init(&s_full, 2);   // the MMA thread, which saw the copies land, and its MMAs
            mbar_init(&s_free, kTcSoft);
            mbar_init(&dp_full, 1);
            mbar_init(&pd_ready, kTcSoft);
            mbar_init(&finished, 1);
            mbar_init(&cleared, 1);
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc(&tmem_base, Sh::kTmemCols);
        tcgen05_fence_before_sync();
    }
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = tmem_base;
    const float *most = p.range.most;
    if (kScaledGradient<T>)
        wait_for_previous_kernel(lse2, delta, bias, most);
    else
        wait_for_previous_kernel(lse2, delta, bias);
    bool ok = true;

    const bool tail = !DKV && cols % kTcN != 0;   // the last tile holds masked keys

    if (warp == kTcCopyWarp) {
        // ---------------------------------------------------- copies
        if (lane == 0 && steps > 0) {
            mbar_arrive_expect_tx(&r_full, 2 * Sh::kRowBytes);
            tc_load<DP, kTcM>(sR1, p.r1, n, h, i0, &r_full);
            tc_load<DP, kTcM>(sR2, p.r2, n, h, i0, &r_full);
            for (int t = 0; t < steps; ++t) {
                const int s = t % NS;
                if (t >= NS) {   // the stage's last tile is consumed
                    ok = tc_wait(&done[s], (t / NS - 1) & 1, a.err);
                    if (!ok) break;
                }
                mbar_arrive_expect_tx(&c_full[s], 2 * Sh::kTileBytes + Sh::kVecBytes +
                                                      (BIAS == kBiasWindow ? p.bias.count * 4 : 0));
                tc_load<DP, kTcN>(sC1 + s * Sh::kTileBytes, p.c1, n, h, t * kTcN, &c_full[s]);
                tc_load<DP, kTcN>(sC2 + s * Sh::kTileBytes, p.c2, n, h, t * kTcN, &c_full[s]);
                if (BIAS == kBiasWindow)
                    bulk_copy_g2s(sBias + s * p.bias.count, bias + bias_start(p.bias, meet(t * kTcN)),
                                  p.bias.count * 4, &c_full[s]);
                if (DKV) {
                    bulk_copy_g2s(sVec + s * 2 * kTcN, lse2 + t * kTcN, kTcN * 4, &c_full[s]);
                    bulk_copy_g2s(sVec + s * 2 * kTcN + kTcN, delta + t * kTcN, kTcN * 4, &c_full[s]);
                }
            }
        }
        __syncwarp();
        if (steps > 0 && tail) {   // what masked keys hold must not reach a product
            const int t = steps - 1;
            ok = tc_wait(&c_full[t % NS], (t / NS) & 1, a.err);
            __syncwarp();
            tc_clear_rows<DP, kTcN>(sC1 + t % NS * Sh::kTileBytes, cols - t * kTcN);
            tc_clear_rows<DP, kTcN>(sC2 + t % NS * Sh::kTileBytes, cols - t * kTcN);
            if (lane == 0) mbar_arrive(&cleared);
        }
        // every copy lands before the block may leave (they have, unless a wait gave up)
        for (int t = max(0, steps - NS); t < steps; ++t)
            tc_wait(&c_full[t % NS], (t / NS) & 1, a.err);
    } else if (warp == kTcMmaWarp) {
        // ---------------------------------------------------- MMAs, one thread
        if (lane == 0 && steps > 0) {
            const uint32_t idesc_s = umma_idesc_f16(kBf16, kTcM, kTcN);
            const int depth = (a.D + 15) / 16;
            const uint32_t idesc_o = umma_idesc_f16_bmn(kBf16, kTcM, depth * 16);
            const uint32_t r1_lo = umma_lo_kmajor(smem_u32(sR1)), r2_lo = umma_lo_kmajor(smem_u32(sR2));
            const uint32_t c1_lo = umma_lo_kmajor(smem_u32(sC1)), c2_lo = umma_lo_kmajor(smem_u32(sC2));
            const uint32_t c1_mn = umma_lo_mnmajor(smem_u32(sC1), kTcN * 128);
            const uint32_t c2_mn = umma_lo_mnmajor(smem_u32(sC2), kTcN * 128);
            constexpr int kTile = Sh::kTileBytes / 16;
            const auto arrived = [&](int t) {   // tile t is in place, masked keys cleared
                return tc_wait(&c_full[t % NS], (t / NS) & 1, a.err) &&
                       (!tail || t + 1 < steps || tc_wait(&cleared, 0, a.err));
            };
            ok = tc_wait(&r_full, 0, a.err) && arrived(0);
            if (ok) {
                tc_scores<DP>(tmem + Sh::kTmemS, r1_lo, c1_lo, idesc_s, depth);
                mbar_arrive(&s_full);
                umma_commit(&s_full);
                tc_scores<DP>(tmem + Sh::kTmemP, r2_lo, c2_lo, idesc_s, depth);
                umma_commit(&dp_full);
            }
            for (int t = 0; t < steps && ok; ++t) {
                const int s = t % NS, s1 = (t + 1) % NS;
                if (t + 1 < steps) {   // the next scores, once this step's are loaded
                    ok = arrived(t + 1) && tc_wait(&s_free, t & 1, a.err);
                    if (!ok) break;
                    tcgen05_fence_after_sync();
                    tc_scores<DP>(tmem + Sh::kTmemS, r1_lo, c1_lo + s1 * kTile, idesc_s, depth);
                    mbar_arrive(&s_full);
                    umma_commit(&s_full);
                }
                ok = tc_wait(&pd_ready, t & 1, a.err);
                if (!ok) break;
                tcgen05_fence_after_sync();
                if (DKV)
                    tc_weighted(tmem + Sh::kTmemAcc2, tmem + Sh::kTmemP, c2_mn + s * kTile, idesc_o,
                                t > 0);
                tc_weighted(tmem + Sh::kTmemAcc1, tmem + Sh::kTmemP + kTcHalf / 2, c1_mn + s * kTile,
                            idesc_o, t > 0);
                umma_commit(t + 1 < steps ? &done[s] : &finished);
                if (t + 1 < steps) {   // p and ds are consumed: dP may be overwritten
                    ok = tc_wait(&done[s], (t / NS) & 1, a.err);
                    if (!ok) break;
                    tc_scores<DP>(tmem + Sh::kTmemP, r2_lo, c2_lo + s1 * kTile, idesc_s, depth);
                    umma_commit(&dp_full);
                }
            }
            if (!ok) {   // a wait gave up: let the MMAs end before TMEM is released
                umma_commit(&r_full);
                tc_wait(&r_full, 1, a.err);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- weights
        // After a wait that gave up a thread goes on without waiting (and its warp
        // without storing), so that its partner finds it at every pair_sync.
        const auto wait = [&](uint64_t *bar, int parity) {
            if (ok) ok = tc_wait(bar, parity, a.err);
            __syncwarp();
        };
        const int pair = warp % 4, part = warp / 4;
        const uint32_t my_tmem = (uint32_t)(pair * 32) << 16;   // this warp's TMEM lanes
        const int first = part * kTcHalf;                       // this thread's columns of a tile
        const int i = i0 + pair * 32 + lane, ic = min(i, live_rows - 1);
        const float c2 = a.scale * kLog2e;
        const int my_row = !BIAS || steps == 0 ? 0 : DKV ? -rel_k(a, ic) : rel_q(a, ic);
        TileWalk walk;
        if (BIAS) walk.init(DKV ? a.Hq : a.Hk, DKV ? a.Wq : a.Wk, a.P);
        const int inverse = 65536 / (DKV ? a.Wq : a.Wk) + 1, meet0 = meet(0);
        const bool counts = i < live_rows && steps > 0;
        const float row_lse = !DKV ? (counts ? lse2[i] : INFINITY) : 0.0f;
        const float row_delta = !DKV && counts ? delta[i] : 0.0f;
        const float up = kScaledGradient<T> ? gradient_scale(most, p.range.parts, nh) : 1.0f;
        const bool with_rel = !DKV && BIAS && p.rel.window > 0 && i0 + pair * 32 < a.Lq && steps > 0;
        RelWindow win;
        float *rel_out = nullptr;
        if (!DKV && BIAS) {
            if (with_rel) rel_out = win.init(a, sRel, p.rel, i0, nh, pair, part);
        }
        int stage = 0;
        // the bias of this row and the next step's first column, and where the
        // thread's columns start in their grid
        const float *row = nullptr;
        int x = 0, rel = 0;
        const auto aim = [&] {
            const int at = meet0 + (DKV ? walk.rel : -walk.rel);
            if (BIAS == kBiasWindow)
                row = sBias + stage * p.bias.count + (at - row0 + my_row - bias_start(p.bias, at));
            else if (BIAS)
                row = bias + at - row0 + my_row;
            if (BIAS) walk.half(part, x, rel);
        };
        aim();
        for (int t = 0; t < steps; ++t) {
            const int live = cols - t * kTcN;
            uint32_t r[kTcHalf], d[kTcHalf];
            float b[kTcHalf];
            wait(&s_full, t & 1);
            tcgen05_fence_after_sync();
            tmem_start_ld_x32(tmem + Sh::kTmemS + my_tmem + first, r);
            constexpr int kSign = DKV ? 1 : -1;
            if (!BIAS) {
#pragma unroll
                for (int c = 0; c < kTcHalf; ++c) b[c] = 0.0f;
            } else if (BIAS == kBiasWindow && p.bias.runs) {
                bias_by_runs<kSign>(row, x, rel, walk, b);
            } else {
                bias_offsets(s_rel[warp], walk, first, live, inverse);
                bias_by_table<kSign>(row, s_rel[warp], b);
            }
            const float *vec = sVec + stage * 2 * kTcN + first;   // lse2 and delta of the columns
            tmem_wait_ld(r);
            tcgen05_fence_before_sync();
            mbar_arrive(&s_free);
            scale_and_bias(r, c2, b);
            if (live < kTcN) {   // columns that do not count, whatever they hold
                asm volatile("" ::: "memory");   // a branch: the selects would cost every tile
#pragma unroll
                for (int c = 0; c < kTcHalf; ++c)
                    if (first + c >= live) r[c] = __float_as_uint(-INFINITY);
            }
            const float2 minus = make_float2(-1.0f, -1.0f);
#pragma unroll
            for (int c = 0; c < kTcHalf; c += 4) {
                float4 e = make_float4(row_lse, row_lse, row_lse, row_lse);
                if (DKV) e = *reinterpret_cast<const float4 *>(vec + c);
                const float2 u = fma_f32x2(make_float2(e.x, e.y), minus,
                                           make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])));
                const float2 v = fma_f32x2(make_float2(e.z, e.w), minus,
                                           make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])));
                r[c] = __float_as_uint(exp2_approx(u.x));
                r[c + 1] = __float_as_uint(exp2_approx(u.y));
                r[c + 2] = __float_as_uint(exp2_approx(v.x));
                r[c + 3] = __float_as_uint(exp2_approx(v.y));
            }
            // the next step's place, among the exponentials
            const int my_rel = with_rel ? walk.rel + walk.offset(min(first + lane, live - 1), inverse) : 0;
            if (BIAS) walk.next();
            if (++stage == NS) stage = 0;
            aim();
            wait(&dp_full, t & 1);
            tcgen05_fence_after_sync();
            tmem_ld_x32(tmem + Sh::kTmemP + my_tmem + first, d);
            float ds[kTcHalf];
#pragma unroll
            for (int c = 0; c < kTcHalf; c += 4) {
                float4 e = make_float4(row_delta, row_delta, row_delta, row_delta);
                if (DKV) e = *reinterpret_cast<const float4 *>(vec + kTcN + c);
                float2 u = fma_f32x2(make_float2(e.x, e.y), minus,
                                     make_float2(__uint_as_float(d[c]), __uint_as_float(d[c + 1])));
                float2 v = fma_f32x2(make_float2(e.z, e.w), minus,
                                     make_float2(__uint_as_float(d[c + 2]), __uint_as_float(d[c + 3])));
                u = mul_f32x2(u, make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])));
                v = mul_f32x2(v, make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])));
                ds[c] = u.x;
                ds[c + 1] = u.y;
                ds[c + 2] = v.x;
                ds[c + 3] = v.y;
            }
            uint32_t w[kTcHalf / 2];
            if (DKV) {
                const float2 up = make_float2(kWeightScale<T>, kWeightScale<T>);
#pragma unroll
                for (int c = 0; c < kTcHalf / 2; ++c) {
                    const float2 e = mul_f32x2(
                        make_float2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), up);
                    w[c] = pack2<T>(e.x, e.y);
                }
                tmem_st_x16(tmem + Sh::kTmemP + my_tmem + first, w);
            }
#pragma unroll
            for (int c = 0; c < kTcHalf / 2; ++c) {
                float2 e = make_float2(ds[2 * c], ds[2 * c + 1]);
                if (kScaledGradient<T>) e = mul_f32x2(e, make_float2(up, up));
                w[c] = pack2<T>(e.x, e.y);
            }
            tmem_st_x16(tmem + Sh::kTmemP + my_tmem + first + kTcHalf / 2, w);
            tmem_wait_st();
            tcgen05_fence_before_sync();
            mbar_arrive(&pd_ready);
            if (!DKV && BIAS) {
                if (with_rel) win.add(ds, live, my_rel, walk.rel, t + 1 == steps, rel_out);
            }
        }
        if (steps > 0) wait(&finished, 0);
        if (__all_sync(0xffffffffu, ok)) {
            tcgen05_fence_after_sync();
            const int64_t at = (((int64_t)n * rows + i) * a.H + h) * a.D;
            for (int which = 0; which < (DKV ? 2 : 1); ++which) {
                T *out = (T *)(which ? p.out2 : p.out1) + at;
                const float f = !counts ? 0.0f : which ? 1.0f / kWeightScale<T> : a.scale / up;
                const uint32_t acc = tmem + (which ? Sh::kTmemAcc2 : Sh::kTmemAcc1) + my_tmem;
#pragma unroll 1
                for (int c = part * 32; c < a.D; c += 64) {   // every other chunk
                    uint32_t o[32];
                    if (steps > 0) {
                        tmem_ld_x32(acc + c, o);
                    }
                    if (i < rows) {
#pragma unroll
                        for (int k = 0; k < 32; k += 8)
                            if (c + k < a.D) {   // D is a multiple of 8
                                uint4 w = make_uint4(0, 0, 0, 0);
                                if (counts) {    // other rows may hold anything
                                    uint32_t *u = &w.x;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        u[e] = pack2<T>(__uint_as_float(o[k + 2 * e]) * f,
                                                        __uint_as_float(o[k + 2 * e + 1]) * f);
                                }
                                *reinterpret_cast<uint4 *>(out + c + k) = w;
                            }
                    }
                }
            }
        }
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == kTcMmaWarp) tmem_dealloc(tmem, Sh::kTmemCols);
}

// The query blocks, then the key blocks: one launch, so that either fills the
// SMs that the other leaves.  The longer ones (the bias gradient) come first: the
// other order takes 126 us instead of 121 at 8 x 8 heads of 32 x 32 tokens; one of
// each in turn takes 155.
template <typename T, int DP, int BIAS>
__global__ void __launch_bounds__(kTcThreads, TcBwdShape<DP, true>::kCtas)
    attn_tc_bwd_kernel(const __grid_constant__ TcBwdArgs kv, const __grid_constant__ TcBwdArgs q,
                       int kv_blocks) {
    const int q_blocks = gridDim.x - kv_blocks;
    if ((int)blockIdx.x < q_blocks)
        attn_tc_bwd_block<T, DP, BIAS, false>(q, blockIdx.x);
    else
        attn_tc_bwd_block<T, DP, BIAS, true>(kv, blockIdx.x - q_blocks);
}

// How a launch reads the bias, and its dynamic shared memory: what the larger of
// the two kinds of blocks needs.
struct TcBwdLaunch {
    int mode, smem;
};
template <int DP> constexpr int tc_bwd_smem(int kv_count, int q_count, int rel_window) {
    using Kv = TcBwdShape<DP, true>;
    using Qs = TcBwdShape<DP, false>;
    return std::max(Kv::kSmem + Kv::kStages * kv_count * 4,
                    Qs::kSmem + rel_smem(rel_window, 4) + Qs::kStages * q_count * 4);
}
static_assert(tc_bwd_smem<128>(0, 0, kRelMost) <= kTcSmemOne, "the bias gradient always fits");
// One mode for both kinds: with a window that is too large for one, or where the
// windows do not fit beside those of the bias gradient (wide heads, a narrow grid of
// queries against a wide one of keys), both read the bias through L1.
template <int DP>
TcBwdLaunch tc_bwd_launch_of(const TcBias &kv, const TcBias &q, bool bias, int rel_window) {
    const int with = tc_bwd_smem<DP>(kv.count, q.count, rel_window);
    if (bias && q.count && kv.count && with <= kTcSmemOne) return {kBiasWindow, with};
    return {bias ? kBiasGlobal : kBiasNone, tc_bwd_smem<DP>(0, 0, rel_window)};
}

template <typename T, int DP, int BIAS>
cudaError_t launch_attn_tc_bwd_as(const TcBwdArgs &kv, const TcBwdArgs &q, int kv_heads, int q_heads,
                                  int smem, cudaStream_t s) {
    auto kernel = attn_tc_bwd_kernel<T, DP, BIAS>;
    static DeviceFlags ready;
    const cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmemOne);
    });
    if (e != cudaSuccess) return e;
    const int kv_blocks = (kv.a.Lk + kTcM - 1) / kTcM * kv_heads;
    const int q_blocks = (q.a.Lq + kTcM - 1) / kTcM * q_heads;
    return launch_next(true, kernel, (unsigned)kv_blocks + (unsigned)q_blocks, kTcThreads, smem, s, kv, q,
                       kv_blocks);
}

// dK and dV of `kv_heads` (batch, head) pairs and dQ of `q_heads` (either may be 0).
template <typename T>
cudaError_t launch_attn_tc_bwd(const TcBwdArgs &kv, const TcBwdArgs &q, int kv_heads, int q_heads,
                               cudaStream_t s) {
    const auto run = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        const TcBwdLaunch as = tc_bwd_launch_of<DP>(kv.bias, q.bias, q.bias.base, q.rel.window);
        return as.mode == kBiasNone ? launch_attn_tc_bwd_as<T, DP, kBiasNone>(kv, q, kv_heads, q_heads, as.smem, s)
               : as.mode == kBiasWindow
                   ? launch_attn_tc_bwd_as<T, DP, kBiasWindow>(kv, q, kv_heads, q_heads, as.smem, s)
                   : launch_attn_tc_bwd_as<T, DP, kBiasGlobal>(kv, q, kv_heads, q_heads, as.smem, s);
    };
    return q.a.D <= 64 ? run(std::integral_constant<int, 64>()) : run(std::integral_constant<int, 128>());
}

}  // namespace gs
