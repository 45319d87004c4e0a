// gs_block_api.cu -- the C ABI of the transformer-block operators (declared in
// include/gs.h): host-side argument checks, then dispatch to the per-dtype
// launchers.  Nothing here allocates, synchronises or throws.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <initializer_list>

#include "../../include/gs.h"
#include "gs_internal.h"

namespace {

constexpr int64_t kMax31 = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxNormWidth = int64_t(1) << 20;
constexpr int64_t kMaxDropout = int64_t(1) << 40;
constexpr int64_t kMaxRelative = int64_t(1) << 24;
constexpr int64_t kMaxHeadWidth = 128;
constexpr int64_t kMaxHeads = 65535;

size_t elem_size(gs_dtype dt) { return dt == GS_F32 ? 4 : 2; }
bool dtype_ok(int dt) { return dt == GS_F32 || dt == GS_F16 || dt == GS_BF16; }
bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// A call's error is its own: the runtime keeps the last one until it is asked for,
// and a later call that asks would take it for its own.
gs_status status_of(cudaError_t e) {
    if (e == cudaSuccess) return GS_OK;
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
}

template <typename F>
gs_status dispatch(gs_dtype dt, F &&f) {
    cudaError_t e;
    switch (dt) {
        case GS_F32: e = f(float()); break;
        case GS_F16: e = f(__half()); break;
        default: e = f(__nv_bfloat16()); break;
    }
    return status_of(e);
}

// a * b <= limit for a, b >= 0 (no overflow).
bool product_fits(int64_t a, int64_t b, int64_t limit) { return a == 0 || b <= limit / a; }

gs_status check_workspace(const void *ws, size_t have, size_t need, size_t align) {
    if (need == 0) return GS_OK;
    if (!ws) return GS_ERR_NULL;
    if (!aligned(ws, align)) return GS_ERR_ALIGN;
    return have < need ? GS_ERR_SHAPE : GS_OK;
}

gs_status check_norm(int64_t rows, int64_t D) {
    return rows < 0 || rows > kMax31 || D < 0 || D > kMaxNormWidth ? GS_ERR_SHAPE : GS_OK;
}

size_t norm_ws_bytes(int64_t rows, int64_t D) {
    return rows == 0 || D == 0
               ? 0
               : (size_t)gs::layer_norm_partial_blocks(rows, D) * 2 * (size_t)D * sizeof(float);
}

// Shapes of an attention call.  *empty: no query, no head or no width at all.
gs_status check_attention(const gs_attention_attrs *at, gs_dtype dt, gs::AttnArgs *a) {
    if (!at) return GS_ERR_NULL;
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    if (!isfinite(at->scale)) return GS_ERR_ATTR;
    if (at->N < 0 || at->H < 0 || at->H > kMaxHeads || at->D < 1 || at->D > kMaxHeadWidth) return GS_ERR_SHAPE;
    for (int d = 0; d < 2; ++d)
        if (at->q_extent[d] < 0 || at->q_extent[d] > kMax31 || at->k_extent[d] < 0 ||
            at->k_extent[d] > kMax31)
            return GS_ERR_SHAPE;
    for (int d = 0; d < 3; ++d)
        if (at->q_strides[d] < 0 || at->k_strides[d] < 0 || at->v_strides[d] < 0)
            return GS_ERR_SHAPE;
    if (!product_fits(at->q_extent[0], at->q_extent[1], kMax31) ||
        !product_fits(at->k_extent[0], at->k_extent[1], kMax31) ||
        !product_fits(at->N, at->H, kMax31))
        return GS_ERR_SHAPE;
    const int64_t Lq = at->q_extent[0] * at->q_extent[1], Lk = at->k_extent[0] * at->k_extent[1];
    if (!product_fits(at->N * at->H, Lq, kMax31) || !product_fits(at->N * at->H, Lk, kMax31))
        return GS_ERR_SHAPE;
    if (at->num_buckets < 0 || !product_fits(at->num_buckets, at->H, kMax31)) return GS_ERR_SHAPE;
    const int64_t rows = at->q_extent[0] + at->k_extent[0] - 1;
    const int64_t cols = at->q_extent[1] + at->k_extent[1] - 1;
    if (Lq > 0 && Lk > 0 && !product_fits(rows, cols, kMaxRelative)) return GS_ERR_SHAPE;
    a->N = (int)at->N;
    a->H = (int)at->H;
    a->D = (int)at->D;
    a->Hq = (int)at->q_extent[0];
    a->Wq = (int)at->q_extent[1];
    a->Hk = (int)at->k_extent[0];
    a->Wk = (int)at->k_extent[1];
    a->Lq = (int)Lq;
    a->Lk = (int)Lk;
    a->P = Lq > 0 && Lk > 0 ? (int)cols : 0;
    a->R = Lq > 0 && Lk > 0 ? (int)(rows * cols) : 0;
    a->nb = (int)at->num_buckets;
    for (int d = 0; d < 3; ++d) {
        a->qs[d] = at->q_strides[d];
        a->ks[d] = at->k_strides[d];
        a->vs[d] = at->v_strides[d];
    }
    a->scale = at->scale;
    a->buckets = nullptr;
    a->k_len = nullptr;
    a->err = nullptr;
    return GS_OK;
}

template <typename F>
size_t by_dtype(gs_dtype dt, F &&f) {
    switch (dt) {
        case GS_F32: return f(float());
        case GS_F16: return f(__half());
        default: return f(__nv_bfloat16());
    }
}

size_t attention_ws(const gs::AttnArgs &a, gs_dtype dt, bool backward) {
    return by_dtype(dt, [&](auto tag) { return gs::attn_ws_bytes<decltype(tag)>(a, backward); });
}

// Nothing to attend with: no query, no key or no head.
bool no_pairs(const gs::AttnArgs &a) { return a.N == 0 || a.H == 0 || a.Lq == 0 || a.Lk == 0; }

// Distance from which bucket e + k of one axis side starts.
int64_t bucket_start(int e, int m, int64_t far, int k) {
    const double at = e * pow((double)far / e, (double)k / (m - e));
    return (int64_t)ceil(at - 1e-9);
}

// Bucket of one axis for a signed offset, query minus key.
int axis_bucket(int64_t offset, int num, int64_t far) {
    const int m = num / 2, e = m / 2;
    const int64_t d = offset < 0 ? -offset : offset;
    int b = (int)d;
    if (d >= e) {   // the last bucket whose start is at most d
        b = e;
        for (int hi = m - 1; b < hi;) {
            const int mid = (b + hi + 1) / 2;
            if (d >= bucket_start(e, m, far, mid - e))
                b = mid;
            else
                hi = mid - 1;
        }
    }
    return b + (offset < 0 ? m : 0);
}

constexpr int64_t kMaxGatedWidth = int64_t(1) << 20;
constexpr int64_t kMaxGatedElements = int64_t(1) << 40;

gs_status check_gated(int64_t rows, int64_t D, int64_t F, int act, gs_dtype dt, gs::GatedArgs *a) {
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    if (act < GS_ACT_SILU || act > GS_ACT_IDENTITY) return GS_ERR_ATTR;
    if (rows < 0 || rows > kMax31 || D < 1 || D > kMaxGatedWidth || F < 0 || F > kMaxGatedWidth ||
        !product_fits(rows, D, kMaxGatedElements) || !product_fits(rows, F, kMaxGatedElements))
        return GS_ERR_SHAPE;
    *a = {rows, (int)D, (int)F, act, nullptr};
    return GS_OK;
}

size_t gated_ws(const gs::GatedArgs &a, gs_dtype dt, bool backward) {
    return by_dtype(dt, [&](auto tag) { return gs::gated_ws_bytes<decltype(tag)>(a, backward); });
}

gs_status check_residual_norm(const gs_residual_norm_attrs *at, gs_dtype dt, gs::ResNormArgs *a) {
    if (!at) return GS_ERR_NULL;
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    if (at->kind != GS_NORM_LAYER && at->kind != GS_NORM_RMS) return GS_ERR_ATTR;
    if (!isfinite(at->alpha) || !(at->epsilon >= 0.0f) || isinf(at->epsilon)) return GS_ERR_ATTR;
    const gs_status st = check_norm(at->rows, at->D);
    if (st != GS_OK) return st;
    if (at->groups < 0 || (at->groups > 0 && at->rows % at->groups != 0) ||
        at->groups > (at->rows > 0 ? at->rows : kMax31))
        return GS_ERR_SHAPE;
    a->rows = at->rows;
    a->D = (int)at->D;
    a->groups = (int)at->groups;
    a->group_rows = at->groups > 0 ? at->rows / at->groups : at->rows;
    a->layer = at->kind == GS_NORM_LAYER;
    a->alpha = at->alpha;
    a->eps = at->epsilon;
    a->err = nullptr;
    return GS_OK;
}

size_t residual_norm_ws(const gs::ResNormArgs &a, gs_dtype dt) {
    if (a.rows == 0 || a.D == 0) return 0;
    return by_dtype(dt, [&](auto tag) { return gs::resnorm_ws_bytes<decltype(tag)>(a); });
}

}  // namespace

extern "C" {

gs_status gs_layer_norm(const void *X, const void *Scale, const void *B, int64_t rows, int64_t D,
                        gs_dtype dt, float epsilon, void *Y, float *Mean, float *InvStdDev,
                        cudaStream_t stream) {
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    const gs_status st = check_norm(rows, D);
    if (st != GS_OK) return st;
    if (!(epsilon >= 0.0f) || isinf(epsilon)) return GS_ERR_ATTR;
    if (rows == 0 || D == 0) return GS_OK;
    if (!X || !Scale || !Y) return GS_ERR_NULL;
    const size_t es = elem_size(dt);
    if (!aligned(X, es) || !aligned(Scale, es) || !aligned(B, es) || !aligned(Y, es) ||
        !aligned(Mean, 4) || !aligned(InvStdDev, 4))
        return GS_ERR_ALIGN;
    const gs::NormArgs a = {rows, (int)D, epsilon};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_layer_norm<decltype(tag)>(X, Scale, B, Y, Mean, InvStdDev, a, stream);
    });
}

gs_status gs_layer_norm_backward_workspace_size(int64_t rows, int64_t D, size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    const gs_status st = check_norm(rows, D);
    if (st == GS_OK) *bytes = norm_ws_bytes(rows, D);
    return st;
}

gs_status gs_layer_norm_backward(const void *dY, const void *X, const void *Scale,
                                 const float *Mean, const float *InvStdDev, int64_t rows,
                                 int64_t D, gs_dtype dt, void *workspace, size_t workspace_bytes,
                                 void *dX, void *dScale, void *dB, cudaStream_t stream) {
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    gs_status st = check_norm(rows, D);
    if (st != GS_OK) return st;
    if (D == 0) return GS_OK;
    if (rows > 0 && (!dY || !X || !Scale || !Mean || !InvStdDev || !dX)) return GS_ERR_NULL;
    const size_t es = elem_size(dt);
    if (!aligned(dY, es) || !aligned(X, es) || !aligned(Scale, es) || !aligned(dX, es) ||
        !aligned(dScale, es) || !aligned(dB, es) || !aligned(Mean, 4) || !aligned(InvStdDev, 4))
        return GS_ERR_ALIGN;
    if (dScale || dB) {
        st = check_workspace(workspace, workspace_bytes, norm_ws_bytes(rows, D), 16);
        if (st != GS_OK) return st;
    }
    const gs::NormArgs a = {rows, (int)D, 0.0f};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_layer_norm_backward<decltype(tag)>(dY, X, Scale, Mean, InvStdDev, dX,
                                                             dScale, dB, (float *)workspace, a,
                                                             stream);
    });
}

gs_status gs_dropout(const void *X, const void *residual, int64_t n, gs_dtype dt, double ratio,
                     uint64_t seed, uint64_t offset, void *Y, cudaStream_t stream) {
    if (!dtype_ok(dt)) return GS_ERR_DTYPE;
    if (n < 0 || n > kMaxDropout) return GS_ERR_SHAPE;
    if (!(ratio >= 0.0 && ratio < 1.0)) return GS_ERR_ATTR;
    if (n == 0) return GS_OK;
    if (!X || !Y) return GS_ERR_NULL;
    const size_t es = elem_size(dt);
    if (!aligned(X, es) || !aligned(residual, es) || !aligned(Y, es)) return GS_ERR_ALIGN;
    const double t = floor(ratio * 4294967296.0 + 0.5);
    const gs::DropoutArgs a = {n, t >= 4294967295.0 ? 0xFFFFFFFFu : (uint32_t)t,
                               (float)(1.0 / (1.0 - ratio)), seed, offset};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_dropout<decltype(tag)>(X, residual, Y, a, stream);
    });
}

gs_status gs_relative_buckets(const int64_t *q_extent, const int64_t *k_extent,
                              const int64_t *q_origin, int num_buckets, int64_t max_distance,
                              int causal, int32_t *buckets, int64_t *count) {
    if (!q_extent || !k_extent || !count) return GS_ERR_NULL;
    *count = 0;
    for (int d = 0; d < 2; ++d)
        if (q_extent[d] < 0 || q_extent[d] > kMax31 || k_extent[d] < 0 || k_extent[d] > kMax31)
            return GS_ERR_SHAPE;
    if (causal != 0 && causal != 1) return GS_ERR_ATTR;
    if (causal && (q_extent[0] > 1 || k_extent[0] > 1)) return GS_ERR_UNSUPPORTED;
    if (num_buckets != 0 && (num_buckets < 4 || num_buckets % 2 || num_buckets > 32768 ||
                             max_distance <= num_buckets / 4))
        return GS_ERR_ATTR;
    if (q_extent[0] == 0 || q_extent[1] == 0 || k_extent[0] == 0 || k_extent[1] == 0) return GS_OK;
    const int64_t rows = q_extent[0] + k_extent[0] - 1, cols = q_extent[1] + k_extent[1] - 1;
    if (!product_fits(rows, cols, kMaxRelative)) return GS_ERR_SHAPE;
    if (!buckets) return GS_ERR_NULL;
    const int64_t oy = q_origin ? q_origin[0] : 0, ox = q_origin ? q_origin[1] : 0;
    const int64_t by_unit = rows > 1 ? (cols > 1 ? num_buckets : 1) : 0;
    *count = num_buckets == 0 ? rows * cols
             : rows > 1 && cols > 1 ? (int64_t)num_buckets * num_buckets
             : rows > 1 || cols > 1 ? num_buckets
                                    : 1;
    for (int64_t r = 0; r < rows; ++r) {
        const int64_t dy = r - (k_extent[0] - 1) + oy;
        const int64_t by = num_buckets && by_unit ? by_unit * axis_bucket(dy, num_buckets, max_distance)
                                                  : 0;
        for (int64_t c = 0; c < cols; ++c) {
            const int64_t dx = c - (k_extent[1] - 1) + ox;
            int64_t b = r * cols + c;
            if (num_buckets) b = by + (cols > 1 ? axis_bucket(dx, num_buckets, max_distance) : 0);
            buckets[r * cols + c] = causal && dx < 0 ? -1 : (int32_t)b;
        }
    }
    return GS_OK;
}

gs_status gs_attention_workspace_size(const gs_attention_attrs *attrs, gs_dtype dt, size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    gs::AttnArgs a;
    const gs_status st = check_attention(attrs, dt, &a);
    if (st == GS_OK && !no_pairs(a)) *bytes = attention_ws(a, dt, false);
    return st;
}

gs_status gs_attention_backward_workspace_size(const gs_attention_attrs *attrs, gs_dtype dt,
                                               size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    gs::AttnArgs a;
    const gs_status st = check_attention(attrs, dt, &a);
    if (st == GS_OK && !no_pairs(a)) *bytes = attention_ws(a, dt, true);
    return st;
}

gs_status gs_attention(const void *Q, const void *K, const void *V, const void *table,
                       const int32_t *buckets, const int32_t *k_len,
                       const gs_attention_attrs *attrs, gs_dtype dt, void *workspace,
                       size_t workspace_bytes, void *O, float *LSE, cudaStream_t stream) {
    gs::AttnArgs a;
    gs_status st = check_attention(attrs, dt, &a);
    if (st != GS_OK) return st;
    if (a.N == 0 || a.H == 0 || a.Lq == 0) return GS_OK;
    if (!Q || !O || (a.Lk > 0 && (!K || !V))) return GS_ERR_NULL;
    if (a.Lk > 0 && a.nb > 0 && (!table || !buckets)) return GS_ERR_NULL;
    if (a.nb == 0 && table) return GS_ERR_SHAPE;
    const size_t es = elem_size(dt);
    if (!aligned(Q, es) || !aligned(K, es) || !aligned(V, es) || !aligned(table, es) ||
        !aligned(O, es) || !aligned(LSE, 4) || !aligned(buckets, 4) || !aligned(k_len, 4))
        return GS_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, no_pairs(a) ? 0 : attention_ws(a, dt, false),
                         256);
    if (st != GS_OK) return st;
    if (a.Lk == 0) a.nb = 0;   // no key: O = 0 and LSE = -inf without a bias
    a.buckets = buckets;
    a.k_len = k_len;
    a.err = gs::device_error_word();
    if (!a.err) return GS_ERR_CUDA;
    const gs::AttnPtrs p = {Q, K, V, table, O, LSE, nullptr, nullptr, nullptr, nullptr, nullptr};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_attn<decltype(tag)>(a, p, workspace, stream);
    });
}

gs_status gs_attention_backward(const void *dO, const void *Q, const void *K, const void *V,
                                const void *O, const float *LSE, const void *table,
                                const int32_t *buckets, const int32_t *k_len,
                                const gs_attention_attrs *attrs, gs_dtype dt, void *workspace,
                                size_t workspace_bytes, void *dQ, void *dK, void *dV,
                                void *dTable, cudaStream_t stream) {
    gs::AttnArgs a;
    gs_status st = check_attention(attrs, dt, &a);
    if (st != GS_OK) return st;
    const bool queries = a.N > 0 && a.H > 0 && a.Lq > 0, keys = a.N > 0 && a.H > 0 && a.Lk > 0;
    if (queries && (!dO || !Q || !O || !LSE || !dQ)) return GS_ERR_NULL;
    if (keys && (!K || !V || !dK || !dV)) return GS_ERR_NULL;
    if (a.nb > 0 && a.H > 0 && !dTable) return GS_ERR_NULL;
    if (queries && keys && a.nb > 0 && (!table || !buckets)) return GS_ERR_NULL;
    if (a.nb == 0 && (table || dTable)) return GS_ERR_SHAPE;
    const size_t es = elem_size(dt);
    if (!aligned(Q, es) || !aligned(K, es) || !aligned(V, es) || !aligned(table, es) ||
        !aligned(O, es) || !aligned(dO, es) || !aligned(dQ, es) || !aligned(dK, es) ||
        !aligned(dV, es) || !aligned(dTable, es) || !aligned(LSE, 4) || !aligned(buckets, 4) ||
        !aligned(k_len, 4))
        return GS_ERR_ALIGN;
    if (no_pairs(a)) {   // every gradient there is is zero
        cudaError_t e = cudaSuccess;
        const auto clear = [&](void *p, int64_t n) {
            if (n > 0 && e == cudaSuccess) e = cudaMemsetAsync(p, 0, (size_t)n * es, stream);
        };
        const int64_t row = (int64_t)a.H * a.D;
        clear(dQ, (int64_t)a.N * a.Lq * row);
        clear(dK, (int64_t)a.N * a.Lk * row);
        clear(dV, (int64_t)a.N * a.Lk * row);
        clear(dTable, (int64_t)a.nb * a.H);
        return status_of(e);
    }
    st = check_workspace(workspace, workspace_bytes, attention_ws(a, dt, true), 256);
    if (st != GS_OK) return st;
    a.buckets = buckets;
    a.k_len = k_len;
    a.err = gs::device_error_word();
    if (!a.err) return GS_ERR_CUDA;
    const gs::AttnPtrs p = {Q,  K,  V,  table, const_cast<void *>(O), const_cast<float *>(LSE),
                            dO, dQ, dK, dV,    dTable};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_attn_backward<decltype(tag)>(a, p, workspace, stream);
    });
}

gs_status gs_gated_linear_workspace_size(int64_t rows, int64_t D, int64_t F, gs_dtype dt,
                                         size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    gs::GatedArgs a;
    const gs_status st = check_gated(rows, D, F, GS_ACT_SILU, dt, &a);
    if (st == GS_OK) *bytes = gated_ws(a, dt, false);
    return st;
}

gs_status gs_gated_linear_backward_workspace_size(int64_t rows, int64_t D, int64_t F, gs_dtype dt,
                                                  size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    gs::GatedArgs a;
    const gs_status st = check_gated(rows, D, F, GS_ACT_SILU, dt, &a);
    if (st == GS_OK) *bytes = gated_ws(a, dt, true);
    return st;
}

gs_status gs_gated_linear(const void *X, const void *Wg, const void *Wu, const void *bg,
                          const void *bu, int64_t rows, int64_t D, int64_t F, gs_activation act,
                          gs_dtype dt, void *workspace, size_t workspace_bytes, void *H, void *G,
                          void *U, cudaStream_t stream) {
    gs::GatedArgs a;
    gs_status st = check_gated(rows, D, F, act, dt, &a);
    if (st != GS_OK) return st;
    if (rows == 0 || F == 0) return GS_OK;
    if (!X || !Wg || !Wu || !H || !bg != !bu || !G != !U) return GS_ERR_NULL;
    const size_t es = elem_size(dt);
    if (!aligned(X, es) || !aligned(Wg, es) || !aligned(Wu, es) || !aligned(bg, es) ||
        !aligned(bu, es) || !aligned(H, es) || !aligned(G, es) || !aligned(U, es))
        return GS_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, gated_ws(a, dt, false), 256);
    if (st != GS_OK) return st;
    a.err = gs::device_error_word();
    if (!a.err) return GS_ERR_CUDA;
    gs::GatedPtrs p = {X, Wg, Wu, bg, bu, H, G, U};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_gated<decltype(tag)>(a, p, workspace, stream);
    });
}

gs_status gs_gated_linear_backward(const void *dH, const void *X, const void *Wg, const void *Wu,
                                   const void *G, const void *U, int64_t rows, int64_t D,
                                   int64_t F, gs_activation act, gs_dtype dt, void *workspace,
                                   size_t workspace_bytes, void *dX, void *dWg, void *dWu,
                                   void *dbg, void *dbu, cudaStream_t stream) {
    gs::GatedArgs a;
    gs_status st = check_gated(rows, D, F, act, dt, &a);
    if (st != GS_OK) return st;
    if (rows > 0 && (!X || !dX)) return GS_ERR_NULL;
    if (F > 0 && (!Wg || !Wu || !dWg || !dWu)) return GS_ERR_NULL;
    if (rows > 0 && F > 0 && (!dH || !G || !U)) return GS_ERR_NULL;
    if (!dbg != !dbu) return GS_ERR_NULL;
    const size_t es = elem_size(dt);
    for (const void *q : {dH, X, Wg, Wu, G, U, (const void *)dX, (const void *)dWg,
                          (const void *)dWu, (const void *)dbg, (const void *)dbu})
        if (!aligned(q, es)) return GS_ERR_ALIGN;
    if (rows == 0 || F == 0) {   // every gradient there is is zero
        cudaError_t e = cudaSuccess;
        const auto clear = [&](void *q, int64_t n) {
            if (q && n > 0 && e == cudaSuccess) e = cudaMemsetAsync(q, 0, (size_t)n * es, stream);
        };
        clear(dX, rows * D);
        clear(dWg, F * D);
        clear(dWu, F * D);
        clear(dbg, F);
        clear(dbu, F);
        return status_of(e);
    }
    st = check_workspace(workspace, workspace_bytes, gated_ws(a, dt, true), 256);
    if (st != GS_OK) return st;
    a.err = gs::device_error_word();
    if (!a.err) return GS_ERR_CUDA;
    gs::GatedPtrs p = {X,  Wg, Wu, nullptr, nullptr, nullptr, const_cast<void *>(G),
                       const_cast<void *>(U), dH, dX, dWg, dWu, dbg, dbu};
    return dispatch(dt, [&](auto tag) {
        return gs::launch_gated_backward<decltype(tag)>(a, p, workspace, stream);
    });
}

gs_status gs_residual_norm(const void *X, const void *Z, const void *gate, const void *z_scale,
                           const void *z_B, const void *Scale, const void *B,
                           const gs_residual_norm_attrs *attrs, gs_dtype dt, void *S, void *Y,
                           float *Stats, cudaStream_t stream) {
    gs::ResNormArgs a;
    const gs_status st = check_residual_norm(attrs, dt, &a);
    if (st != GS_OK) return st;
    if (a.rows == 0 || a.D == 0) return GS_OK;
    if (!X || !Z || !Scale || !S || !Y || (a.groups > 0 && !gate) || (z_B && !z_scale))
        return GS_ERR_NULL;
    if (a.groups == 0 && gate) return GS_ERR_SHAPE;
    const size_t es = elem_size(dt);
    for (const void *q : {X, Z, gate, z_scale, z_B, Scale, B, (const void *)S, (const void *)Y})
        if (!aligned(q, es)) return GS_ERR_ALIGN;
    if (!aligned(Stats, 16)) return GS_ERR_ALIGN;
    gs::ResNormPtrs p = {};
    p.gate = gate;
    p.z_scale = z_scale;
    p.z_B = z_B;
    p.scale = Scale;
    p.B = B;
    p.X = X;
    p.Z = Z;
    p.S = S;
    p.Y = Y;
    p.stats = Stats;
    return dispatch(dt, [&](auto tag) { return gs::launch_resnorm<decltype(tag)>(a, p, stream); });
}

gs_status gs_residual_norm_backward_workspace_size(const gs_residual_norm_attrs *attrs,
                                                   gs_dtype dt, size_t *bytes) {
    if (!bytes) return GS_ERR_NULL;
    *bytes = 0;
    gs::ResNormArgs a;
    const gs_status st = check_residual_norm(attrs, dt, &a);
    if (st == GS_OK) *bytes = residual_norm_ws(a, dt);
    return st;
}

gs_status gs_residual_norm_backward(const void *dS, const void *dY, const void *S, const void *Z,
                                    const float *Stats, const void *gate, const void *z_scale,
                                    const void *z_B, const void *Scale,
                                    const gs_residual_norm_attrs *attrs, gs_dtype dt,
                                    void *workspace, size_t workspace_bytes, void *dX, void *dZ,
                                    void *dgate, void *dz_scale, void *dz_B, void *dScale,
                                    void *dB, cudaStream_t stream) {
    gs::ResNormArgs a;
    gs_status st = check_residual_norm(attrs, dt, &a);
    if (st != GS_OK) return st;
    if (a.D == 0) return GS_OK;
    if (a.rows > 0 && (!dY || !S || !Z || !Stats || !Scale || !dX || !dZ)) return GS_ERR_NULL;
    if (a.groups > 0 && ((a.rows > 0 && !gate) || !dgate)) return GS_ERR_NULL;
    if (!z_scale && (z_B || dz_scale || dz_B)) return GS_ERR_NULL;
    if (a.groups == 0 && (gate || dgate)) return GS_ERR_SHAPE;
    const size_t es = elem_size(dt);
    for (const void *q : {dS, dY, S, Z, gate, z_scale, z_B, Scale, (const void *)dX,
                          (const void *)dZ, (const void *)dgate, (const void *)dz_scale,
                          (const void *)dz_B, (const void *)dScale, (const void *)dB})
        if (!aligned(q, es)) return GS_ERR_ALIGN;
    if (!aligned(Stats, 16)) return GS_ERR_ALIGN;
    st = check_workspace(workspace, workspace_bytes, residual_norm_ws(a, dt), 256);
    if (st != GS_OK) return st;
    a.err = gs::device_error_word();
    if (!a.err) return GS_ERR_CUDA;
    if (a.rows == 0 && a.groups > 0) {   // gates of no row
        const gs_status done = status_of(
            cudaMemsetAsync(dgate, 0, (size_t)a.groups * a.D * es, stream));
        if (done != GS_OK) return done;
    }
    gs::ResNormPtrs p = {};
    p.gate = gate;
    p.z_scale = z_scale;
    p.z_B = z_B;
    p.scale = Scale;
    p.Z = Z;
    p.S = const_cast<void *>(S);
    p.stats = const_cast<float *>(Stats);
    p.dS = dS;
    p.dY = dY;
    p.dX = dX;
    p.dZ = dZ;
    p.dgate = dgate;
    p.dz_scale = dz_scale;
    p.dz_B = dz_B;
    p.dScale = dScale;
    p.dB = dB;
    return dispatch(dt, [&](auto tag) {
        return gs::launch_resnorm_backward<decltype(tag)>(a, p, workspace, stream);
    });
}

}  // extern "C"
