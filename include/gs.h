/*
 * gs.h -- C ABI of libgs, GB300 (sm_103a) kernels for spatial-transformer
 * sampling: AffineGrid, GridSample, the two fused, and DeformConv; and for the
 * transformer block over the sampled tokens: layer norm, dropout, attention with a
 * relative position bias, the gated projections of a feed-forward half and the
 * norms around a gated branch, with their gradients.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are caller-owned, dense, row-major (C-contiguous) DEVICE buffers
 *    in the operators' layouts.  Shapes and attributes are HOST values.
 *  - One dtype per call: theta, X, grid, W, offset, B, mask and Y all use
 *    `dt`.  Arithmetic is fp32 (coordinates in exact fixed point, see
 *    gs_grid_sample); half types are widened on load and rounded to nearest
 *    even on store.
 *  - The library allocates no memory, keeps no state between calls and never
 *    synchronises: every call only enqueues kernels on `stream` (0 = the
 *    legacy default stream) and returns.  Scratch space, where a path uses
 *    some, is a workspace the caller passes in, or (gs_grid_sample_static) a
 *    fixed array in the library's static device memory.  Output buffers must
 *    not overlap inputs.
 *  - Arguments are checked on the host before anything is enqueued; a bad
 *    argument returns its gs_status and leaves the outputs untouched.  A
 *    failed launch returns GS_ERR_CUDA.  A tensor with a zero extent is valid
 *    and returns GS_OK without a launch.  Nothing throws across the ABI.
 *  - Pointers must be aligned to their element size (GS_ERR_ALIGN).
 *  - Limits (GS_ERR_SHAPE beyond them): each spatial extent <= 2^20; each
 *    (n, c) slab of X or Y < 2^31 elements; batch and channel counts < 2^31.
 *  - Host threads may call the library at the same time.  The only host-side
 *    state is per-device setup done on the first call that needs it (a
 *    kernel's shared-memory limit, a symbol's device address); it is kept in
 *    atomics, and two threads that both run it get the same result.  Calls
 *    whose outputs overlap race on the device, as any two kernels would, and
 *    so do overlapping gs_grid_sample_static calls (one scratch).
 */
#ifndef GS_H
#define GS_H

#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GS_OK = 0,
    GS_ERR_NULL = 1,        /* a required pointer is NULL                          */
    GS_ERR_RANK = 2,        /* spatial rank r not supported by this entry point    */
    GS_ERR_SHAPE = 3,       /* extents inconsistent, negative or beyond the limits */
    GS_ERR_DTYPE = 4,       /* unknown gs_dtype                                    */
    GS_ERR_ATTR = 5,        /* unknown mode / padding, bad kernel/stride/group ... */
    GS_ERR_ALIGN = 6,       /* a pointer is not aligned to its element size        */
    GS_ERR_CUDA = 7,        /* the CUDA runtime reported an error at launch        */
    GS_ERR_TIMEOUT = 8,     /* a bounded device-side wait gave up (see gs_device_status) */
    GS_ERR_UNSUPPORTED = 9  /* valid by the operator spec, not implemented here    */
} gs_status;

typedef enum { GS_F32 = 0, GS_F16 = 1, GS_BF16 = 2 } gs_dtype;

/* GridSample - version 20, Attributes, mode.  The version-16 names "bilinear"
 * and "bicubic" are the same modes (the Python binding maps them). */
typedef enum { GS_LINEAR = 0, GS_NEAREST = 1, GS_CUBIC = 2 } gs_mode;

/* GridSample - version 20, Attributes, padding_mode. */
typedef enum { GS_PAD_ZEROS = 0, GS_PAD_BORDER = 1, GS_PAD_REFLECTION = 2 } gs_pad;

/*
 * gs_affine_grid -- AffineGrid (ai.onnx, since version 20): description and
 * Inputs/Outputs.
 *
 *   theta  device, (N, r, r+1): the affine matrices without their implicit
 *          last row [0 .. 0 1].
 *   r      2 or 3.
 *   size   host, r+2 int64: (N, C, H, W) or (N, C, D, H, W); C is unused.
 *   align_corners  0: -1 and 1 are the outer edges of the corner pixels, the
 *          base positions are (2i+1)/n - 1; 1: they are the corner pixel
 *          centres, -1 + 2i/(n-1) (an axis of length 1 sits at 0).
 *   grid   device output, (N, H, W, 2) or (N, D, H, W, 3); each vector lists
 *          the width coordinate first.  Computed in fp64, rounded once.
 */
gs_status gs_affine_grid(const void *theta, gs_dtype dt, int r, const int64_t *size,
                         int align_corners, void *grid, cudaStream_t stream);

/*
 * gs_grid_sample -- GridSample - version 20 (and version 22): description,
 * Inputs, Outputs and Attributes.
 *
 *   X        device, (N, C, D1..Dr): values at pixel centres.
 *   x_shape  host, r+2 int64.
 *   r        1 to 6 spatial dimensions (GS_ERR_RANK otherwise).
 *   grid     device, (N, D1_out..Dr_out, r); the location vector lists the
 *            innermost axis first (x -> width, y -> height, z -> depth).
 *   out_spatial  host, r int64: D1_out..Dr_out.
 *   mode     linear (N-linear), nearest (ties to the even index), cubic
 *            (N-cubic, Keys kernel with coefficient cubic_coeff_a).
 *   pad      zeros: out-of-range taps read 0; border: clamp; reflection:
 *            mirror at the borders until in range, then clamp.  For linear
 *            and nearest the coordinate is padded; for cubic each tap index is.
 *   align_corners  as in gs_affine_grid: x = (g+1)/2*(n-1) for 1,
 *            x = ((g+1)*n - 1)/2 for 0.
 *   cubic_coeff_a  Keys' a (the operator uses -0.75); ignored unless cubic.
 *   Y        device output, (N, C, D1_out..Dr_out).
 *
 * The unnormalised coordinate is formed without rounding error (an exact
 * product split, then 32.32 fixed point), so nearest picks the same index as
 * exact arithmetic, ties included.  Ranks 4 to 6 run on one rank-general
 * kernel (the tap product summed axis by axis, innermost first); the
 * operator's description defines any rank r, and 6 is this library's limit.
 *
 * Speed: this call reads X in its own NCHW layout, one 2- or 4-byte load per
 * tap and channel.  Grids with spatial locality (smooth warps) are served well
 * from L2; random-access 2-D grids are not, since every tap of every channel
 * then touches its own 32-byte sector.  For those, gs_grid_sample_ws (or
 * gs_grid_sample_static) copies X to channel-last order first and reads each
 * tap as 16-byte runs of channels; on a 16 x 64 x 256^2 fp32 image batch with
 * a uniformly random cubic grid it is about five times faster, copy included.
 */
gs_status gs_grid_sample(const void *X, const int64_t *x_shape, int r, const void *grid,
                         const int64_t *out_spatial, gs_dtype dt, gs_mode mode, gs_pad pad,
                         int align_corners, float cubic_coeff_a, void *Y, cudaStream_t stream);

/*
 * gs_grid_sample_workspace_size -- device workspace that gs_grid_sample_ws
 * asks for with these shapes: whole image slots, a slot being (H*W + 1) * C
 * elements of `dt`, enough for the batch in equal chunks of at most about
 * 512 MB (at least one slot).  0 means the call never uses a workspace (rank
 * other than 2, C * element size not a multiple of 16 bytes,
 * (H*W + 1) * C >= 2^31, or an empty tensor).  Arguments as gs_grid_sample;
 * `bytes` is a host output.  Shape errors are reported as by gs_grid_sample.
 */
gs_status gs_grid_sample_workspace_size(const int64_t *x_shape, int r, const int64_t *out_spatial,
                                        gs_dtype dt, size_t *bytes);

/*
 * gs_grid_sample_ws -- gs_grid_sample with a caller-owned device workspace
 * (GridSample - version 20, as above; the same results, value for value).
 *
 *   workspace        device, 16-byte aligned (GS_ERR_ALIGN), or NULL.
 *   workspace_bytes  its size.  With room for one image slot ((H*W + 1) * C
 *                    elements of `dt`: a zero pixel, then the image), 2-D
 *                    calls copy X to channel-last order there, as many whole
 *                    images at a time as it holds, then read every tap as
 *                    16-byte runs of channels: for grids without spatial
 *                    locality this cuts the bytes read per output several
 *                    fold.  Each chunk costs a copy launch and a sampling
 *                    launch, so fewer, larger chunks are faster.  With less
 *                    than one slot, or NULL, it is gs_grid_sample.
 *
 * The workspace's contents on entry do not matter and are garbage on return.
 * Calls on different streams must not share a workspace while in flight.
 */
gs_status gs_grid_sample_ws(const void *X, const int64_t *x_shape, int r, const void *grid,
                            const int64_t *out_spatial, gs_dtype dt, gs_mode mode, gs_pad pad,
                            int align_corners, float cubic_coeff_a, void *workspace,
                            size_t workspace_bytes, void *Y, cudaStream_t stream);

/* Integer element types of X for gs_grid_sample_int. */
typedef enum { GS_U8 = 16, GS_I8 = 17, GS_U16 = 18, GS_I16 = 19 } gs_itype;

/*
 * gs_grid_sample_int -- GridSample - version 20 with an integer-typed X
 * (Type Constraints, T1; Outputs: "for integer input types, intermediate
 * values are computed as floating point and cast to integer at the end").
 *
 *   X, Y     device, integer type `xt` (uint8, int8, uint16, int16), the
 *            layouts of gs_grid_sample.
 *   grid     device, floating type `grid_dt` (T2: float, float16; bfloat16
 *            as in version 22).
 *   Other arguments, and the taps and weights, as gs_grid_sample.
 *
 * X is widened to fp32 (exact for these types), interpolated in fp32, then
 * truncated toward zero and saturated at the range of `xt` (cubic weights can
 * overshoot it).  Errors as gs_grid_sample; GS_ERR_DTYPE for another `xt` or
 * `grid_dt`.
 */
gs_status gs_grid_sample_int(const void *X, gs_itype xt, const int64_t *x_shape, int r,
                             const void *grid, gs_dtype grid_dt, const int64_t *out_spatial,
                             gs_mode mode, gs_pad pad, int align_corners, float cubic_coeff_a,
                             void *Y, cudaStream_t stream);

/* Size of the scratch gs_grid_sample_static uses: 64 MiB per device. */
#define GS_STATIC_WORKSPACE_BYTES (64u << 20)

/*
 * gs_grid_sample_static -- gs_grid_sample_ws whose workspace is a fixed
 * GS_STATIC_WORKSPACE_BYTES array in the library's static device memory, so
 * the call allocates nothing (no cudaMalloc, no allocating library call) and
 * needs no caller buffer.  It is meant for callers that cannot allocate
 * device memory at the point of the call: a plugin inside a host framework
 * that owns all device memory through its own pool and hands out only
 * inputs and outputs; a real-time loop that must not block, since
 * cudaMalloc and cudaFree can synchronise the device; or code whose memory
 * budget is fixed at start-up, where an allocation failing mid-run has no
 * way to recover.  The operator pages have no counterpart to this call; it
 * wraps the same kernels as gs_grid_sample_ws.
 *
 *   Arguments, results and errors as gs_grid_sample.  A call the channel-
 *   last path takes (see gs_grid_sample_workspace_size) whose image slot,
 *   (H*W + 1) * C elements of `dt`, exceeds GS_STATIC_WORKSPACE_BYTES
 *   returns GS_ERR_SHAPE before anything is enqueued; other calls run the
 *   NCHW gather and touch no scratch.
 *
 * The scratch needs no clearing: each call writes every byte it reads.  The
 * first call on each device looks up the scratch's address (and the error
 * word's) once with cudaGetSymbolAddress, GS_ERR_CUDA if that fails: make it
 * before any stream capture.  There is one scratch per device and process:
 * calls in flight at the same time on different streams, or from different
 * host threads, race on it and corrupt each other's results.
 */
gs_status gs_grid_sample_static(const void *X, const int64_t *x_shape, int r, const void *grid,
                                const int64_t *out_spatial, gs_dtype dt, gs_mode mode, gs_pad pad,
                                int align_corners, float cubic_coeff_a, void *Y,
                                cudaStream_t stream);

/*
 * gs_affine_sample -- GridSample(X, AffineGrid(theta, size)) in one kernel
 * (AffineGrid, ai.onnx since version 20: description, Inputs and Outputs;
 * GridSample - version 20: description, Inputs and Attributes): the grid is
 * generated per output position in registers and never touches memory (the
 * spatial transformer's grid generator and sampler).
 *
 *   theta    device, (N, r, r+1).
 *   size     host, r+2 int64: (N, C, out...), AffineGrid's size input; N and
 *            C must equal X's.
 *   X, x_shape, mode, pad, align_corners, cubic_coeff_a, Y: as gs_grid_sample,
 *            with Y (N, C, out...).  align_corners applies to both operators.
 *
 * The grid is not rounded to `dt` between the two operators.  Positions are
 * affine in the output index; the kernel evaluates that map in 64-bit fixed
 * point (coefficients from fp64), so an identity theta reproduces X exactly.
 */
gs_status gs_affine_sample(const void *theta, const int64_t *size, int r, const void *X,
                           const int64_t *x_shape, gs_dtype dt, gs_mode mode, gs_pad pad,
                           int align_corners, float cubic_coeff_a, void *Y,
                           cudaStream_t stream);

/*
 * gs_affine_sample_from_host -- gs_affine_sample with theta, X and Y in host
 * memory: the batch is cut into `chunks` runs of whole images, and for each
 * run the upload of theta and X (streams[0]), the kernel (streams[1]) and the
 * download of Y (streams[2]) are enqueued with cudaMemcpyAsync and ordered by
 * events, so the copies of neighbouring runs overlap the kernels.  The
 * operator is independent per image, so the result equals gs_affine_sample's
 * bit for bit.
 *
 *   theta_h, X_h, Y_h     host; page-locked (cudaHostAlloc / cudaHostRegister)
 *                         for the copies to overlap, pageable works but
 *                         serialises them.  Y_h is written.
 *   theta_d, X_d, Y_d     device buffers of the full sizes (caller-owned; the
 *                         library allocates nothing), aligned as gs_affine_sample
 *                         wants X, theta and Y.
 *   chunks                runs to cut the batch into (clamped to [1, N]).
 *   streams               host, three caller-owned streams: upload, kernel,
 *                         download.  Nothing orders them against other work:
 *                         make streams[0] wait for whatever produced theta_h
 *                         and X_h, and wait on streams[2] before reading Y_h.
 *   Other arguments as gs_affine_sample.
 *
 * Errors as gs_affine_sample; GS_ERR_NULL for a missing host or device buffer
 * or stream array; GS_ERR_CUDA if a copy, event or launch fails to enqueue
 * (runs already enqueued stay enqueued).
 */
gs_status gs_affine_sample_from_host(const void *theta_h, const int64_t *size, int r,
                                     const void *X_h, const int64_t *x_shape, gs_dtype dt,
                                     gs_mode mode, gs_pad pad, int align_corners,
                                     float cubic_coeff_a, void *Y_h, void *theta_d, void *X_d,
                                     void *Y_d, int chunks, const cudaStream_t *streams);

/*
 * DeformConv attributes.  The DeformConv page lists no Attributes section; its
 * examples use kernel_shape, pads and offset_group.  The rest follow ONNX Conv:
 *   kernel     (kH, kW); 0 means "take it from W".
 *   pads       (top, left, bottom, right).
 *   strides    (sH, sW), >= 1.     dilations (dH, dW), >= 1.
 *   group      C and oC divisible by it.
 *   offset_group  C divisible by it.
 * Output extents: oH = (H + top + bottom - dH*(kH-1) - 1) / sH + 1, same for W.
 */
typedef struct {
    int64_t kernel[2], pads[4], strides[2], dilations[2], group, offset_group;
} gs_deform_attrs;

/*
 * gs_deform_conv -- DeformConv (ai.onnx, since version 22), 2-D: Inputs and
 * Outputs.
 *
 *   X       device, (N, C, H, W).        x_shape host, 4 int64.
 *   W       device, (oC, C/group, kH, kW).
 *   oC      output channels.
 *   offset  device, (N, offset_group*kH*kW*2, oH, oW): for offset group o and
 *           kernel position k = kh*kW + kw, channel o*2K + 2k is the row (y)
 *           offset and o*2K + 2k + 1 the column (x) offset, K = kH*kW.
 *   B       device, (oC), or NULL for zeros.
 *   mask    device, (N, offset_group*kH*kW, oH, oW), or NULL for ones.
 *   Y       device output, (N, oC, oH, oW).
 *
 * Each sample is bilinear in X at (oh*sH - top + kh*dH + dy,
 * ow*sW - left + kw*dW + dx); taps outside X read 0.  fp32 contracts with
 * fp32 FMAs; bf16 and fp16 contract the sampled column tile on the tensor
 * cores where the shape allows (fp32 accumulation), else with fp32 FMAs.
 */
gs_status gs_deform_conv(const void *X, const int64_t *x_shape, const void *W, int64_t oC,
                         const void *offset, const void *B, const void *mask,
                         const gs_deform_attrs *attrs, gs_dtype dt, void *Y,
                         cudaStream_t stream);

/*
 * gs_deform_conv_workspace_size -- device workspace gs_deform_conv_ws asks
 * for: the packed W (rounded up to 256 bytes) and one channel-last slot of
 * (H*W + 1) * C elements per image.  0 means the call never uses a
 * workspace: fp32, or a shape outside the tensor-core path (group or
 * offset_group > 1, C or oC not a multiple of 16, oC > 256, or W too large
 * for shared memory).  Arguments as gs_deform_conv (no tensors needed);
 * `bytes` is a host output.
 */
gs_status gs_deform_conv_workspace_size(const int64_t *x_shape, int64_t oC,
                                        const gs_deform_attrs *attrs, gs_dtype dt, size_t *bytes);

/*
 * gs_deform_conv_ws -- gs_deform_conv with a caller-owned device workspace
 * (DeformConv, as above; the same values).
 *
 *   workspace        device, 256-byte aligned (GS_ERR_ALIGN), or NULL.
 *   workspace_bytes  its size.  With room for the packed W and at least one
 *                    image slot, fp16/bf16 calls on the tensor-core path pack
 *                    W once, copy X to channel-last order (as many images at a
 *                    time as it holds) and read each bilinear tap as 16-byte
 *                    runs of channels.  Otherwise it is gs_deform_conv.
 *
 * The workspace's contents on entry do not matter and are garbage on return.
 * Calls on different streams must not share a workspace while in flight.
 */
gs_status gs_deform_conv_ws(const void *X, const int64_t *x_shape, const void *W, int64_t oC,
                            const void *offset, const void *B, const void *mask,
                            const gs_deform_attrs *attrs, gs_dtype dt, void *workspace,
                            size_t workspace_bytes, void *Y, cudaStream_t stream);

/*
 * Resize -- Resize - 18 (Summary, Attributes, Inputs) on the same separable
 * sampler.  Attribute values follow the operator's names.
 */
typedef enum {
    GS_RS_HALF_PIXEL = 0, GS_RS_PYTORCH_HALF_PIXEL = 1, GS_RS_ALIGN_CORNERS = 2,
    GS_RS_ASYMMETRIC = 3, GS_RS_TF_CROP_AND_RESIZE = 4
} gs_resize_coord;
typedef enum {
    GS_RS_ROUND_PREFER_FLOOR = 0, GS_RS_ROUND_PREFER_CEIL = 1, GS_RS_FLOOR = 2, GS_RS_CEIL = 3
} gs_resize_nearest;
typedef enum { GS_RS_STRETCH = 0, GS_RS_NOT_LARGER = 1, GS_RS_NOT_SMALLER = 2 } gs_resize_keep;

typedef struct {
    gs_mode mode;                  /* nearest (the operator's default), linear, cubic      */
    gs_resize_coord coord;         /* coordinate_transformation_mode, default half_pixel   */
    gs_resize_nearest nearest_mode;/* default round_prefer_floor                           */
    float cubic_coeff_a;           /* default -0.75                                        */
    int exclude_outside;           /* 0 or 1                                               */
    float extrapolation_value;     /* tf_crop_and_resize outside the input                 */
    int antialias;                 /* 0 or 1: stretch linear / cubic by 1/scale downscaling */
    gs_resize_keep keep_aspect_ratio_policy;   /* applies to sizes                         */
} gs_resize_attrs;

/*
 * gs_resize_output_shape -- output extents of Resize (host only).
 *
 *   rank, x_shape  host: X's rank (1..8) and extents.
 *   axes, naxes    host: the axes scales / sizes / roi refer to (negative
 *                  counts from the back), or NULL / 0 for all axes in order.
 *   scales         host float[naxes or rank], > 0, or NULL.  Output extent
 *                  floor(in * (roi_end - roi_start) * scale).
 *   sizes          host int64[naxes or rank], >= 0, or NULL.  Exactly one of
 *                  scales and sizes.  keep_aspect_ratio_policy not_larger /
 *                  not_smaller take one common scale, min / max of
 *                  sizes[i] / in[axes[i]], and round scale * in halfway up.
 *   roi            host float[2 * (naxes or rank)]: starts then ends,
 *                  normalised; used only with tf_crop_and_resize (NULL: 0..1).
 *   y_shape        host output, rank int64.
 * Errors: GS_ERR_NULL, GS_ERR_RANK, GS_ERR_SHAPE (bad extents, repeated axis),
 * GS_ERR_ATTR (bad attribute, scale <= 0, both or neither of scales/sizes).
 */
gs_status gs_resize_output_shape(int rank, const int64_t *x_shape, const int64_t *axes, int naxes,
                                 const float *scales, const int64_t *sizes, const float *roi,
                                 const gs_resize_attrs *attrs, int64_t *y_shape);

/*
 * gs_resize -- Resize - 18 of X into Y (device buffers, `dt` for both).
 * Arguments as gs_resize_output_shape; Y must have that shape.
 *
 * Each axis maps output index o to x_original by the coordinate
 * transformation (with "scales" the given scale is used and the resized
 * length is n * scale, unfloored; with "sizes" scale = out / in), then takes
 * its taps: nearest (nearest_mode), linear (floor(x), floor(x) + 1), cubic
 * (floor(x) - 1 .. floor(x) + 2, Keys with cubic_coeff_a); antialias stretches
 * the linear / cubic filter by 1/scale when downscaling and rescales the
 * weights to sum 1; taps outside the axis read the edge value, or get weight
 * 0 with the rest rescaled when exclude_outside = 1.  The output is the sum
 * over the tensor product of the taps of the weights' product times X;
 * tf_crop_and_resize writes extrapolation_value wherever x_original leaves
 * [0, n - 1] on any axis.  Coordinates are formed in fp64; values accumulate
 * in fp32.
 *
 * Axes whose map is the identity (same extent, scale 1, whole roi) are
 * batched; the resized ones must be the last three or fewer
 * (GS_ERR_UNSUPPORTED otherwise), with at most 64 taps per output index
 * (antialias down to scale ~1/16 cubic, ~1/32 linear).
 */
gs_status gs_resize(const void *X, int rank, const int64_t *x_shape, const int64_t *axes,
                    int naxes, const float *scales, const int64_t *sizes, const float *roi,
                    const gs_resize_attrs *attrs, gs_dtype dt, void *Y, cudaStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators of a transformer block over sampled tokens.  A sampled map or
 * glimpse is a grid of tokens; these calls normalise them, let them attend to
 * one another with a learned bias by relative grid position, and drop and sum
 * the branch, each with its gradient.  Sums, statistics, running maxima and
 * accumulators are fp32.  No sum depends on the order in which threads finish: a
 * call repeated on the same inputs gives the same bits.
 *
 * Layer norm and dropout round once, at the store, and so does attention in fp32,
 * in 16-bit types whose rows are not multiples of 16 bytes, and forward for up to
 * eight queries.  Elsewhere the tensor cores take fp16 and bf16, and the factors
 * of the second products are rounded to the type as well: the softmax weights
 * (forward, and for dV) and their gradients dS (for dQ and dK), half a step of the
 * type on every term.  Results are then off by 2.0e-3 to 2.4e-3 of their size in
 * bf16 and by 3e-4 in fp16, where the store alone is 1.7e-3 and 2e-4.  In fp16 the
 * weights are scaled by a power of two, and dS by one that the largest rows of dO
 * and V allow, so that neither leaves the type's range.  Attention's exponential
 * is the hardware's (ex2.approx.ftz), in fp32 too.
 * ---------------------------------------------------------------------------
 */

/*
 * gs_layer_norm -- LayerNormalization (ai.onnx, since version 17): Inputs X,
 * Scale, B; Attributes epsilon; Outputs Y, Mean, InvStdDev (stash_type 1).
 *
 *   X        device, (rows, D): the axes from `axis` on are flattened into D.
 *   Scale    device, (D).          B  device, (D), or NULL for zeros.
 *   rows     < 2^31.               D  <= 2^20.
 *   epsilon  >= 0, added to the variance.
 *   Y        device output, (rows, D).
 *   Mean, InvStdDev  device outputs, (rows) fp32, or NULL.  The backward pass
 *            takes both.
 *
 * mean = sum x / D, var = sum (x - mean)^2 / D (two passes over the row, held
 * on chip up to D = 8192), InvStdDev = 1 / sqrt(var + epsilon),
 * Y = (x - mean) * InvStdDev * Scale + B.  With D = 0 nothing is written.
 */
gs_status gs_layer_norm(const void *X, const void *Scale, const void *B, int64_t rows, int64_t D,
                        gs_dtype dt, float epsilon, void *Y, float *Mean, float *InvStdDev,
                        cudaStream_t stream);

/* Device workspace gs_layer_norm_backward needs (host output `bytes`). */
gs_status gs_layer_norm_backward_workspace_size(int64_t rows, int64_t D, size_t *bytes);

/*
 * gs_layer_norm_backward -- the gradient of gs_layer_norm.
 *
 *   dY       device, (rows, D).     X, Scale, Mean, InvStdDev as above.
 *   workspace  device, 16-byte aligned (GS_ERR_ALIGN), at least the size
 *            gs_layer_norm_backward_workspace_size reports (GS_ERR_SHAPE for
 *            less, GS_ERR_NULL for none) unless dScale and dB are both NULL.
 *   dX       device output, (rows, D).
 *   dScale, dB  device outputs, (D) of `dt`, each or both NULL.  With rows = 0
 *            they are written as zeros.
 *
 * xhat = (x - Mean) * InvStdDev, g = dY * Scale,
 * dX = InvStdDev * (g - mean(g) - xhat * mean(g * xhat)),
 * dScale = sum over rows of dY * xhat, dB = sum over rows of dY.
 */
gs_status gs_layer_norm_backward(const void *dY, const void *X, const void *Scale,
                                 const float *Mean, const float *InvStdDev, int64_t rows,
                                 int64_t D, gs_dtype dt, void *workspace, size_t workspace_bytes,
                                 void *dX, void *dScale, void *dB, cudaStream_t stream);

/*
 * gs_dropout -- Dropout (ai.onnx, since version 13) in training mode, with an
 * optional residual sum: Y = residual + (kept ? X / (1 - ratio) : 0).
 *
 *   X, residual, Y  device, n elements; residual may be NULL.  Y may be X or
 *            residual itself (in place); other overlaps are not allowed.
 *   n        <= 2^40.
 *   ratio    in [0, 1): the probability of dropping, to 2^-32.
 *   seed, offset  the generator's key and stream.  Take another offset for
 *            every layer and step.
 *
 * Element i draws word i % 4 of Philox4x32-10 (Salmon et al., SC 2011) with
 * key `seed` and counter (i / 4, offset), low words first, and is kept when
 * word >= round(ratio * 2^32), 2^32 - 1 at most.  The mask is a function of these numbers alone
 * and is stored nowhere.  The gradient with respect to X is the same call on
 * dY (no residual) with the same ratio, seed and offset; the gradient with
 * respect to the residual is dY.
 */
gs_status gs_dropout(const void *X, const void *residual, int64_t n, gs_dtype dt, double ratio,
                     uint64_t seed, uint64_t offset, void *Y, cudaStream_t stream);

/*
 * Shapes of gs_attention.  Queries lie on a grid of q_extent = (Hq, Wq) tokens
 * and keys on one of k_extent = (Hk, Wk), both row-major, Lq = Hq * Wq and
 * Lk = Hk * Wk; a plain sequence is (1, L).
 *   N, H, D     batch, heads (at most 65535), head width (1 to 128).
 *   *_strides   strides of Q, K and V in elements for (batch, token, head);
 *               the D elements of a head are contiguous.  This covers
 *               (N, L, H, D) and (N, H, L, D) tensors, a packed
 *               (N, L, 3, H, D) projection and heads that share keys (stride
 *               0).  O, dO, dQ, dK and dV are dense (N, L, H, D).
 *   num_buckets rows of the bias table, or 0 for no bias.
 *   scale       of the scores, usually 1 / sqrt(D); finite.
 * Limits (GS_ERR_SHAPE): extents and strides >= 0, N * H * Lq and N * H * Lk
 * < 2^31, (Hq+Hk-1) * (Wq+Wk-1) <= 2^24, num_buckets * H < 2^31.
 */
typedef struct {
    int64_t N, H, D;
    int64_t q_extent[2], k_extent[2];
    int64_t q_strides[3], k_strides[3], v_strides[3];
    int64_t num_buckets;
    float scale;
} gs_attention_attrs;

/*
 * gs_relative_buckets -- a bucket map for gs_attention (host only).
 *
 *   q_extent, k_extent  host, the two grids.
 *   q_origin   host, the key-grid position of query (0, 0), or NULL for
 *              (0, 0): one new token at the end of a sequence of L keys has
 *              q_extent (1, 1) and q_origin (0, L - 1).
 *   num_buckets  buckets per axis, or 0 to give every relative position its
 *              own.  Otherwise even, >= 4 (a multiple of 2 whose half has a
 *              first half): per axis, half of the buckets belong to keys at or
 *              before the query (offset query - key >= 0) and half to keys
 *              after it; in each, the first half hold one distance each and
 *              the rest grow by a constant ratio: with m = num_buckets / 2 and
 *              e = m / 2, bucket e + k starts at distance
 *              ceil(e * (max_distance / e)^(k / (m - e))).  The last of them,
 *              k = m - e - 1, takes every distance from its start on;
 *              max_distance is where one more would start (16 buckets and a
 *              max_distance of 64: the last holds 32 and up).
 *              An axis on which both grids have extent 1 takes no part; with
 *              two axes the bucket is by * num_buckets + bx.
 *   max_distance  > num_buckets / 4.
 *   causal     0, or 1: keys after the query in token order of the key grid
 *              get -1, which masks them.  Needs grids of one row
 *              (GS_ERR_UNSUPPORTED otherwise).
 *   buckets    host output, (Hq+Hk-1) * (Wq+Wk-1) int32.
 *   count      host output: rows the bias table needs.
 */
gs_status gs_relative_buckets(const int64_t *q_extent, const int64_t *k_extent,
                              const int64_t *q_origin, int num_buckets, int64_t max_distance,
                              int causal, int32_t *buckets, int64_t *count);

/* Device workspace gs_attention and gs_attention_backward need (host output
 * `bytes`; 0: none). */
gs_status gs_attention_workspace_size(const gs_attention_attrs *attrs, gs_dtype dt, size_t *bytes);
gs_status gs_attention_backward_workspace_size(const gs_attention_attrs *attrs, gs_dtype dt,
                                               size_t *bytes);

/*
 * gs_attention -- softmax attention with a learned bias by relative position.
 *
 *   Q, K, V   device, (N, Lq | Lk, H, D) through their strides.
 *   table     device, (num_buckets, H) of `dt`, or NULL with num_buckets = 0.
 *   buckets   device, (Hq+Hk-1, Wq+Wk-1) int32: entry
 *             (yq - yk + Hk-1, xq - xk + Wk-1) names the pair's row of the
 *             table.  A value outside [0, num_buckets) masks the pair, and so
 *             does a table entry of -inf (causal and local attention are
 *             bucket maps).  A masked pair has the weight 0, but its K and V
 *             are read: what is not finite there may make the row NaN.
 *   k_len     device, (N) int32, or NULL: keys from k_len[n] on are masked
 *             (clamped to [0, Lk]); what K and V hold there is never used.
 *             The items share the map, and with it the queries' place among
 *             the keys: a new token that stands at the end of its own item's
 *             keys takes a call per item where items end at different lengths.
 *   workspace device, 256-byte aligned (GS_ERR_ALIGN), at least the size
 *             gs_attention_workspace_size reports (GS_ERR_NULL for none,
 *             GS_ERR_SHAPE for less).
 *   O         device output, (N, Lq, H, D).
 *   LSE       device output, (N, H, Lq) fp32, or NULL: the natural logarithm
 *             of the sum of exponentials, which the backward pass takes.
 *
 * s = scale * q . k + table[bucket][h];  O = softmax(s) V.  A row whose mask
 * leaves no key gives O = 0 and LSE = -inf.  A row of finite entries as low as
 * the type allows is an ordinary softmax.  Scores are held in base 2 in fp32: a
 * finite table entry beyond +-2.35e38 counts as that, in O and in LSE.
 *
 * LSE is one fp32 number, and the weights that the backward pass forms from it
 * are as good as its spacing: to 2^-9 where it is near -1e4, to one half near
 * -1e6.  In a row whose scores are all of the size of -1e9 and below, where it
 * holds nothing of their number, the largest scores have the weight 1 each, not
 * 1 / count.  Where the gradients of such rows matter, mask the pairs by an entry
 * of -inf or a bucket outside the table, whose rows have none.
 */
gs_status gs_attention(const void *Q, const void *K, const void *V, const void *table,
                       const int32_t *buckets, const int32_t *k_len,
                       const gs_attention_attrs *attrs, gs_dtype dt, void *workspace,
                       size_t workspace_bytes, void *O, float *LSE, cudaStream_t stream);

/*
 * gs_attention_backward -- the gradient of gs_attention.
 *
 *   dO, O     device, (N, Lq, H, D).       LSE  device, (N, H, Lq) fp32.
 *   dQ, dK, dV  device outputs, dense (N, Lq | Lk, H, D).  Rows of masked keys
 *             and of queries with no key are zero.  dO is read in every row: one
 *             that is not finite reaches dK and dV, and dQ's row, with no key too.
 *   dTable    device output, (num_buckets, H) of `dt`; NULL without a table.
 *   Other arguments as gs_attention; the workspace's size is
 *   gs_attention_backward_workspace_size.
 *
 * With p = exp(s - LSE) and delta = dO . O per query:
 * dS = p * (dO . v - delta);  dQ = scale * dS K;  dK = scale * dS^T Q;
 * dV = p^T dO;  dTable[b][h] = sum of dS over the batch and bucket b's pairs.
 */
gs_status gs_attention_backward(const void *dO, const void *Q, const void *K, const void *V,
                                const void *O, const float *LSE, const void *table,
                                const int32_t *buckets, const int32_t *k_len,
                                const gs_attention_attrs *attrs, gs_dtype dt, void *workspace,
                                size_t workspace_bytes, void *dQ, void *dK, void *dV,
                                void *dTable, cudaStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * The feed-forward half of the block: its gated projections, and the norms on both
 * sides of a branch with the branch's gate and the scaled residual sum.
 * ---------------------------------------------------------------------------
 */

/* Activation of the gated projections: g / (1 + e^-g); g Phi(g) with the normal
 * distribution's Phi; its tanh form 0.5 g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)));
 * max(g, 0); 1 / (1 + e^-g); g. */
typedef enum {
    GS_ACT_SILU = 0, GS_ACT_GELU = 1, GS_ACT_GELU_TANH = 2, GS_ACT_RELU = 3, GS_ACT_SIGMOID = 4,
    GS_ACT_IDENTITY = 5
} gs_activation;

/* Device workspace gs_gated_linear and gs_gated_linear_backward need (host output
 * `bytes`; 0: none), with or without biases. */
gs_status gs_gated_linear_workspace_size(int64_t rows, int64_t D, int64_t F, gs_dtype dt,
                                         size_t *bytes);
gs_status gs_gated_linear_backward_workspace_size(int64_t rows, int64_t D, int64_t F, gs_dtype dt,
                                                  size_t *bytes);

/*
 * gs_gated_linear -- both projections of a gated feed-forward block, the activation
 * and the product: G = X Wg^T + bg, U = X Wu^T + bu, H = act(G) * U.
 *
 *   X         device, (rows, D).
 *   Wg, Wu    device, (F, D): an output's weights are contiguous.
 *   bg, bu    device, (F), or both NULL.
 *   rows      < 2^31.      D, F  1 <= D <= 2^20, F <= 2^20; rows * D and rows * F
 *             <= 2^40.
 *   workspace device, 256-byte aligned (GS_ERR_ALIGN), at least the size
 *             gs_gated_linear_workspace_size reports (GS_ERR_NULL for none,
 *             GS_ERR_SHAPE for less).
 *             Calls that may run at the same time, replays of captured graphs among
 *             them, need one each; calls in order on a stream may share one.
 *   H         device output, (rows, F).
 *   G, U      device outputs, (rows, F), both or neither: what the backward pass
 *             takes.
 *
 * The sums over D are fp32; G, U and H are each rounded once, at the store, and H
 * is formed of the unrounded G and U.  Up to 16 rows need no workspace, nor up to 32
 * with F < 4864 (rows of more than 2^18 16-bit elements aside).
 *
 * fp32, more rows than those: each factor is taken as three bf16 numbers, and six of their
 * products are summed in fp32; that keeps fp32's precision, but of a factor below about
 * 2^-110 the lowest bits are lost, and a factor that is infinite, or two whose product
 * leaves fp32's range, may give NaN where a plain sum gives an infinity.
 * The activations take hardware approximations of the exponential and the reciprocal
 * (2 ulps each), whose argument is rounded: 1 / (1 + e^-g) is off by up to |g| 2^-23 of
 * itself more, Phi and its density by 1.5 g^2 2^-24.  Phi is a polynomial times e^(-g^2/2),
 * off by 1.1e-6 of itself in 16-bit types and 7e-9 in fp32.  Where 1 / (1 + e^-g) or Phi is
 * below 2^-126 it counts as 0.
 * More rows than those of a 16-bit type run on plain FMAs, 7 to 50 times slower, where
 * D > 32768, or where D is a multiple of 8 and X, Wg or Wu starts on no 16-byte boundary.
 */
gs_status gs_gated_linear(const void *X, const void *Wg, const void *Wu, const void *bg,
                          const void *bu, int64_t rows, int64_t D, int64_t F, gs_activation act,
                          gs_dtype dt, void *workspace, size_t workspace_bytes, void *H, void *G,
                          void *U, cudaStream_t stream);

/*
 * gs_gated_linear_backward -- the gradient of gs_gated_linear.
 *
 *   dH, G, U  device, (rows, F).
 *   dX        device output, (rows, D).      dWg, dWu  device outputs, (F, D).
 *   dbg, dbu  device outputs, (F), or both NULL.
 *   Other arguments as gs_gated_linear; the workspace's size is
 *   gs_gated_linear_backward_workspace_size.
 *
 * dG = dH * U * act'(G), dU = dH * act(G); dX = dG Wg + dU Wu; dWg = dG^T X,
 * dWu = dU^T X; dbg and dbu are the sums of dG and dU over the rows.  relu's slope
 * at 0 is 0.  In 16-bit types dG and dU are rounded to the type as factors of the
 * products (half a step on every term); the biases' sums take them unrounded.  In
 * fp16 they are scaled by a power of two before that rounding, from the largest finite
 * |dG| or |dU| of the call, and the products are scaled back: neither a scaled loss nor
 * a small one leaves the type's range.  Elements below 2^-28 of the largest are off by
 * up to 2^-39 of it, where others are off by half a step; what is below that may count
 * as 0.  A value that is not finite stays in its row of dX and its output's rows of dWg
 * and dWu.  With rows = 0 the gradients of the weights and biases are zeros.
 */
gs_status gs_gated_linear_backward(const void *dH, const void *X, const void *Wg, const void *Wu,
                                   const void *G, const void *U, int64_t rows, int64_t D,
                                   int64_t F, gs_activation act, gs_dtype dt, void *workspace,
                                   size_t workspace_bytes, void *dX, void *dWg, void *dWu,
                                   void *dbg, void *dbu, cudaStream_t stream);

/* The norms of gs_residual_norm: (x - mean) / sqrt(var + epsilon), or
 * x / sqrt(mean(x^2) + epsilon). */
typedef enum { GS_NORM_LAYER = 0, GS_NORM_RMS = 1 } gs_norm_kind;

/*
 * Shapes of gs_residual_norm.
 *   rows    < 2^31.      D  <= 2^20.
 *   groups  rows of the gate, or 0 without one; it divides `rows`.  rows / groups
 *           consecutive rows share one: 1 is a gate per channel, the batch's items a
 *           gate for each, `rows` one for every row.
 *   kind    of both norms.
 *   alpha   factor of the residual, finite.     epsilon  >= 0.
 */
typedef struct {
    int64_t rows, D, groups;
    gs_norm_kind kind;
    float alpha, epsilon;
} gs_residual_norm_attrs;

/*
 * gs_residual_norm -- the norm after a branch, its gate, the scaled residual sum and
 * the norm before the next branch, in one pass:
 *   z' = norm(Z) * z_scale + z_B, or Z without z_scale,
 *   S = alpha * X + gate * z',   Y = norm(S) * Scale + B.
 *
 *   X, Z      device, (rows, D): the residual and the branch's output.
 *   gate      device, (groups, D), or NULL with groups = 0 (a factor of 1).
 *   z_scale   device, (D), or NULL for no norm of Z.
 *   z_B, B    device, (D), or NULL for zeros; z_B needs z_scale (GS_ERR_NULL).
 *   Scale     device, (D).
 *   S, Y      device outputs, (rows, D).  Y is formed of the unrounded S.
 *   Stats     device output, (rows, 4) fp32, 16-byte aligned, or NULL: the mean and
 *             the reciprocal deviation of Z (0 and 1 without z_scale) and those of S
 *             (means are 0 for GS_NORM_RMS).  The backward pass takes them.
 */
gs_status gs_residual_norm(const void *X, const void *Z, const void *gate, const void *z_scale,
                           const void *z_B, const void *Scale, const void *B,
                           const gs_residual_norm_attrs *attrs, gs_dtype dt, void *S, void *Y,
                           float *Stats, cudaStream_t stream);

/* Device workspace gs_residual_norm_backward needs (host output `bytes`). */
gs_status gs_residual_norm_backward_workspace_size(const gs_residual_norm_attrs *attrs,
                                                   gs_dtype dt, size_t *bytes);

/*
 * gs_residual_norm_backward -- the gradient of gs_residual_norm.
 *
 *   dS        device, (rows, D), or NULL for zeros: what reaches S otherwise.
 *   dY        device, (rows, D).
 *   S, Stats  the forward pass's.
 *   dX, dZ    device outputs, (rows, D).
 *   dgate     device output, (groups, D); NULL without a gate.
 *   dz_scale, dz_B, dScale, dB  device outputs, (D), each or all NULL; dz_scale and
 *             dz_B need z_scale.  With rows = 0 they are written as zeros.
 *   workspace device, 256-byte aligned, at least the size
 *             gs_residual_norm_backward_workspace_size reports.
 *             Calls that may run at the same time, replays of captured graphs among
 *             them, need one each; calls in order on a stream may share one.
 *
 * With N(w, x^, inv) = inv * (w - mean(w) - x^ * mean(w * x^)) (no mean(w) for
 * GS_NORM_RMS), s^ and z^ the normalised S and Z:
 * ds = dS + N(dY * Scale, s^, inv_s);  dX = alpha * ds;  dScale = sum dY * s^,
 * dB = sum dY;  dgate = sum of ds * z' over the rows that share it;  e = gate * ds;
 * dz_scale = sum e * z^, dz_B = sum e;  dZ = N(e * z_scale, z^, inv_z), or e.
 * The sums over rows are taken in an order that shapes and alignment decide: the same
 * call gives the same bits.  Above D = 4096 with a gate or z_scale, and above 8192, the
 * inputs are read twice.
 */
gs_status gs_residual_norm_backward(const void *dS, const void *dY, const void *S, const void *Z,
                                    const float *Stats, const void *gate, const void *z_scale,
                                    const void *z_B, const void *Scale,
                                    const gs_residual_norm_attrs *attrs, gs_dtype dt,
                                    void *workspace, size_t workspace_bytes, void *dX, void *dZ,
                                    void *dgate, void *dz_scale, void *dz_B, void *dScale,
                                    void *dB, cudaStream_t stream);

/* Human-readable name of a status code (static storage). */
const char *gs_status_str(gs_status s);

/*
 * gs_device_status -- synchronises `stream`, then reports (and clears) the
 * library's device-side error word: GS_ERR_TIMEOUT if a bounded wait inside a
 * kernel gave up since the last call, GS_ERR_CUDA if the stream holds a CUDA
 * error, else GS_OK.  Kernels that give up a wait stop early and leave their
 * output incomplete; they never trap.
 */
gs_status gs_device_status(cudaStream_t stream);

/*
 * gs_test_bounded_wait_expires -- a test hook, not an operator (no page
 * defines it).  Enqueues one kernel on `stream` in which a single thread arms
 * an mbarrier for 16 bytes of transfer that no copy will ever deliver, then
 * waits on it with the same bounded wait the pipelined kernels use, with a
 * limit of `limit_ns` nanoseconds of the GPU's global timer.  The wait runs
 * out, records GS_ERR_TIMEOUT in the device error word and the kernel
 * returns, so a test can check that path without breaking a pipeline: the
 * next gs_device_status reports GS_ERR_TIMEOUT (and clears it).  Nothing is in
 * flight when the kernel leaves, so the context stays usable.  `limit_ns`
 * must lie in [1, 1e9] (GS_ERR_ATTR otherwise); nothing is allocated.
 */
gs_status gs_test_bounded_wait_expires(uint64_t limit_ns, cudaStream_t stream);

/* Library version, "major.minor.patch" (static storage). */
const char *gs_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GS_H */
