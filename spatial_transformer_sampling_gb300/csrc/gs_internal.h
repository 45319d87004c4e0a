// gs_internal.h -- host-side interface between the C ABI (gs_api.cu) and the
// per-dtype kernel translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace gs {

// Host-side per-device setup (a kernel's shared-memory attribute, a symbol's
// device address) runs on the first call that needs it on each device.  The
// flags are atomics, so first calls from several host threads at once do not
// race on them; the setup steps are idempotent, so two such calls may both run
// a step and both get the same result.
constexpr int kMaxDevices = 64;

struct DeviceFlags {
    std::atomic<bool> set[kMaxDevices];
};

// Runs setup() unless it already succeeded on the current device; returns its
// error (cudaSuccess once done).
template <typename F>
cudaError_t once_per_device(DeviceFlags &flags, F &&setup) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && flags.set[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = setup();
    if (e == cudaSuccess && cached) flags.set[dev].store(true, std::memory_order_release);
    return e;
}

// Launches a kernel of a call whose kernels follow one another.  With `follows` it
// comes after one of the same call: its blocks are set up once that one's blocks
// have ended, and it waits by itself (wait_for_previous_kernel) for what that one
// wrote before it reads or writes anything that the two share: 3 us less per pair
// of kernels.  (Set up while the earlier kernel's blocks still run, they spread
// unevenly over the SMs: attention over 1500 tokens, 6 heads, fp32, 242 us and not
// 160.)  Every kernel in between waits too, so that the end of one means the end
// of all before it; a call's first kernel is launched without, so that nothing of
// the call runs before the stream's earlier work has ended.
struct LaunchAs {
    bool follows;
    int cluster;   // blocks of a cluster, along x
    LaunchAs(bool follows_, int cluster_ = 1) : follows(follows_), cluster(cluster_) {}
};
template <typename... P, typename... A>
cudaError_t launch_next(LaunchAs as, void (*kernel)(P...), dim3 grid, int threads, int smem,
                        cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2];
    cfg.attrs = attrs;
    if (as.follows) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (as.cluster > 1) {
        attrs[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attrs[cfg.numAttrs].val.clusterDim.x = (unsigned)as.cluster;
        attrs[cfg.numAttrs].val.clusterDim.y = attrs[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

constexpr int kSampleThreads = 256;

struct Axis;   // gs_common.cuh

// Arguments of the sampling kernels (GridSample and the fused affine path).
// Largest spatial rank GridSample takes (ranks 4 and up run on one
// rank-general kernel; the fused and channel-last paths take ranks 2 and 3).
constexpr int kMaxRankND = 6;

struct SampleArgs {
    int N, C;
    int in[kMaxRankND];  // input spatial extents, outermost first (1 when unused)
    int out[kMaxRankND]; // output spatial extents, outermost first
    int64_t in_plane;    // product of in[]
    int64_t out_plane;   // product of out[]
    int tiles;           // blocks per image: ceil(out_plane / kSampleThreads)
    int pad, ac;
    float a;             // Keys coefficient
    unsigned *err;       // device error word (bounded waits record timeouts here)
};

// Arguments of the standalone AffineGrid kernel.
struct AffineGridArgs {
    int N;
    int out[3];
    int64_t out_plane;
    int ac;
};

// Arguments of DeformConv.
struct DeformArgs {
    int N, C, H, W, oC, oH, oW;
    int kH, kW, pad_t, pad_l, sH, sW, dH, dW, group, offset_group;
    int has_bias, has_mask;
    unsigned *err;       // device error word (bounded waits record timeouts here)
};

// Resize (Resize - 18): coordinate maps and nearest rounding.
enum { RS_HALF_PIXEL = 0, RS_PYTORCH_HALF_PIXEL = 1, RS_ALIGN_CORNERS = 2, RS_ASYMMETRIC = 3,
       RS_TF_CROP_AND_RESIZE = 4 };
enum { RS_ROUND_PREFER_FLOOR = 0, RS_ROUND_PREFER_CEIL = 1, RS_FLOOR = 2, RS_CEIL = 3 };

// One resized axis.  taps: taps per output index (1 nearest, 2 linear,
// 4 cubic, more when antialiasing a downscale); k0: offset of the first tap
// from floor(x) (the last is 1 - k0); aa_scale: the scale the filter is
// stretched by (1 unless antialiasing a downscale).
struct ResizeAxis {
    int n_in, n_out;
    double scale, length_resized, roi_start, roi_end, aa_scale;
    int k0, taps;
};

constexpr int kRsMaxTapsHost = 64;   // taps per output index the Resize kernel holds

// Arguments of the Resize kernel: r trailing resized axes in ax[3-r..2]
// (ax[0..2-r] are unit axes), B slices made of the leading axes.
struct ResizeArgs {
    ResizeAxis ax[3];
    int64_t B;
    int r;
    int mode, coord, nearest_mode;
    double a;
    int exclude_outside;
    float extrapolation_value;
    unsigned *err;   // device error word (bounded waits record timeouts here)
};

// Per-dtype launchers; T is float, __half or __nv_bfloat16.  Each enqueues on
// `s` and returns the launch error (cudaSuccess when fine).
// `ws`, `ws_bytes`: optional device workspace for the channel-last GridSample
// path (NULL, or fewer bytes than one image: the NCHW gather runs instead).
template <typename T>
cudaError_t launch_sample(const void *X, const void *src, void *Y, const SampleArgs &args, int r,
                          int mode, bool affine, void *ws, size_t ws_bytes, cudaStream_t s);
// Workspace bytes the channel-last path asks for (0: this call never takes it),
// and the least it runs with (one image slot).
template <typename T>
size_t sample_workspace_bytes(const SampleArgs &args, int r, bool affine);
template <typename T>
size_t sample_min_workspace_bytes(const SampleArgs &args);
template <typename T>
cudaError_t launch_affine_grid(const void *theta, void *grid, const AffineGridArgs &args, int r,
                               cudaStream_t s);
template <typename T>
cudaError_t launch_deform(const void *X, const void *W, const void *offset, const void *B,
                          const void *mask, void *Y, const DeformArgs &args, cudaStream_t s);
// DeformConv with an optional workspace for the channel-last tensor-core path
// (too small or NULL: launch_deform), and the workspace bytes that path asks
// for (0: it never takes the shape).
template <typename T>
cudaError_t launch_deform_ws(const void *X, const void *W, const void *offset, const void *B,
                             const void *mask, void *Y, const DeformArgs &args, void *ws,
                             size_t ws_bytes, cudaStream_t s);
template <typename T>
size_t deform_ws_bytes(const DeformArgs &args);
// DeformConv (fp16 / bf16) on the staged persistent tensor-core kernel
// (gs_deform_st.cuh) when it takes the shape and pointers; *used reports
// whether it ran.  deform_staged_takes answers the same question.
template <typename T>
cudaError_t launch_deform_staged(const void *X, const void *W, const void *offset, const void *B,
                                 const void *mask, void *Y, const DeformArgs &args, cudaStream_t s,
                                 bool *used);
bool deform_staged_takes(const DeformArgs &args, const void *X, const void *W, const void *offset,
                         const void *mask);
// DeformConv (fp32) on the windowed register-tiled kernel (gs_deform_f32.cu)
// when it takes the shape and X pointer; *used reports whether it ran.
cudaError_t launch_deform_f32(const void *X, const void *W, const void *offset, const void *B,
                              const void *mask, void *Y, const DeformArgs &args, cudaStream_t s,
                              bool *used);
bool deform_f32_takes(const DeformArgs &args, const void *X);
template <typename T>
cudaError_t launch_resize(const void *X, void *Y, const ResizeArgs &args, cudaStream_t s);
// GridSample with integer X (TX: uint8_t, int8_t, uint16_t, int16_t) and a float
// grid of gs_dtype code `grid_dt`.
template <typename TX>
cudaError_t launch_sample_int(const void *X, const void *grid, int grid_dt, void *Y,
                              const SampleArgs &args, int r, int mode, cudaStream_t s);

// ------------------------------------------------ transformer-block operators

// Device address of the library's error word on the current device.
unsigned *device_error_word();

// Layer norm over the last axis of `rows` x `D` elements (gs_norm.cu).
struct NormArgs {
    int64_t rows;
    int D;
    float eps;
};
template <typename T>
cudaError_t launch_layer_norm(const void *X, const void *scale, const void *B, void *Y, float *mean,
                              float *inv, const NormArgs &args, cudaStream_t s);
template <typename T>
cudaError_t launch_layer_norm_backward(const void *dY, const void *X, const void *scale,
                                       const float *mean, const float *inv, void *dX, void *dScale,
                                       void *dB, float *partials, const NormArgs &args,
                                       cudaStream_t s);
// Row blocks whose column sums the backward pass keeps apart: it needs
// 2 * blocks * D floats of workspace.
int layer_norm_partial_blocks(int64_t rows, int64_t D);

// Dropout with an optional residual sum over `n` elements (gs_dropout.cu).
struct DropoutArgs {
    int64_t n;
    uint32_t threshold;      // a word below it drops its element
    float scale;             // 1 / (1 - ratio)
    uint64_t seed, offset;
};
template <typename T>
cudaError_t launch_dropout(const void *X, const void *residual, void *Y, const DropoutArgs &args,
                           cudaStream_t s);

// Attention with a relative position bias (gs_attn*.cu).  Token i of the
// queries sits at (i / Wq, i % Wq) of its grid, token j of the keys at
// (j / Wk, j % Wk); the pair's relative index is
//   rel_q(i) - rel_k(j),  rel_q(i) = yi * P + xi + (Hk-1) * P + Wk-1,
//   rel_k(j) = yj * P + xj,  P = Wq + Wk - 1,
// in [0, R), R = (Hq+Hk-1) * P.
struct AttnArgs {
    int N, H, D;
    int Hq, Wq, Hk, Wk, Lq, Lk, P, R;
    int nb;                             // rows of the bias table (0: no bias)
    int bias_stride;                    // floats per head of the expanded bias
    int64_t qs[3], ks[3], vs[3];        // strides of batch, token, head in elements
    float scale;                        // of the scores
    const int *buckets;                 // device (R) or nullptr
    const int *k_len;                   // device (N) or nullptr
    unsigned *err;
};
struct AttnPtrs {                       // device pointers; backward only from dO on
    const void *Q, *K, *V, *table;
    void *O;
    float *lse;
    const void *dO;
    void *dQ, *dK, *dV, *dTable;
};
// Workspace bytes (a multiple of 256) of the forward and backward calls.
template <typename T> size_t attn_ws_bytes(const AttnArgs &args, bool backward);
template <typename T>
cudaError_t launch_attn(const AttnArgs &args, const AttnPtrs &p, void *ws, cudaStream_t s);
template <typename T>
cudaError_t launch_attn_backward(const AttnArgs &args, const AttnPtrs &p, void *ws,
                                 cudaStream_t s);

// Gated projections of a feed-forward block (gs_gated*.cu).
struct GatedArgs {
    int64_t rows;
    int D, F;
    int act;                            // gs_activation
    unsigned *err;
};
struct GatedPtrs {                      // device pointers; forward: G and U are outputs
    const void *X, *Wg, *Wu, *bg, *bu;
    void *H, *G, *U;
    const void *dH;
    void *dX, *dWg, *dWu, *dbg, *dbu;
};
template <typename T> size_t gated_ws_bytes(const GatedArgs &args, bool backward);
template <typename T>
cudaError_t launch_gated(const GatedArgs &args, const GatedPtrs &p, void *ws, cudaStream_t s);
template <typename T>
cudaError_t launch_gated_backward(const GatedArgs &args, const GatedPtrs &p, void *ws,
                                  cudaStream_t s);

// Norms around a gated branch (gs_residual_norm.cuh).
struct ResNormArgs {
    int64_t rows;
    int D;
    int groups;                         // rows of the gate, 0 without one
    int64_t group_rows;                 // rows that share one
    int layer;                          // layer norms: means are subtracted
    float alpha, eps;
    unsigned *err;
};
struct ResNormPtrs {                    // device pointers
    const void *gate, *z_scale, *z_B, *scale, *B;
    const void *X, *Z;
    void *S, *Y;
    float *stats;
    const void *dS, *dY;                // backward: S is an input, B unused
    void *dX, *dZ, *dgate, *dz_scale, *dz_B, *dScale, *dB;
};
template <typename T> size_t resnorm_ws_bytes(const ResNormArgs &args);
template <typename T>
cudaError_t launch_resnorm(const ResNormArgs &args, const ResNormPtrs &p, cudaStream_t s);
template <typename T>
cudaError_t launch_resnorm_backward(const ResNormArgs &args, const ResNormPtrs &p, void *ws,
                                    cudaStream_t s);

}  // namespace gs
