// gs_attn_tc.cuh -- tensor-core building blocks of the attention kernels
// (fp16 / bf16): tiles staged by TMA with the 128-byte swizzle, tcgen05.mma
// with both operands in shared memory or the first in tensor memory (TMEM),
// and the TMEM loads and stores the softmax warps use.
//
// A tile of R tokens holds DP / 64 chunks of R rows x 128 bytes (64 elements
// of the head width; what lies beyond D arrives as zeros).  The same bytes
// serve as a K-major operand (contraction over the head width: scores) and as
// an MN-major one (contraction over tokens: the weighted sums), so nothing is
// transposed in memory.
#pragma once

#include <limits.h>

#include <type_traits>

#include "gs_attn_rel.cuh"
#include "gs_ptx.cuh"
#include "gs_tma.cuh"

namespace gs {

constexpr int kTcM = 128;            // rows of a score tile, two softmax threads each
constexpr int kTcN = 64;             // columns of a score tile
constexpr int kTcHalf = kTcN / 2;    // columns of one softmax thread
constexpr int kTcSoft = 2 * kTcM;    // softmax threads: warps w and w + 4 share rows 32 (w % 4) on
constexpr int kTcThreads = kTcSoft + 64;   // and a warp that issues MMAs, and one that copies
constexpr int kTcMmaWarp = kTcSoft / 32, kTcCopyWarp = kTcMmaWarp + 1;

// mbar_wait_bounded for waits on the critical path of a pipeline: polls without
// reading the global timer, which takes longer than the events waited for, but
// for every 1024th poll.
__device__ __forceinline__ bool tc_wait(uint64_t *bar, uint32_t parity, unsigned *err) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
        if (n % 1024 != 0) continue;
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            atomicOr(err, kDevErrTimeout);
            return false;
        }
    }
    return true;
}

// Barrier of the two warps that share 32 rows.
__device__ __forceinline__ void pair_sync(int pair) {
    asm volatile("bar.sync %0, 64;" ::"r"(pair + 1) : "memory");
}

// The same barrier; true for all of its 64 threads when `p` is for any.
__device__ __forceinline__ bool pair_any(int pair, bool p) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %2, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(pair + 1), "r"((uint32_t)p)
        : "memory");
    return any != 0;
}

// Shared-memory descriptors with the 128-byte swizzle (see
// umma_desc_kmajor_sw128): the upper word is the same for all of a kernel's
// operands (1024 bytes between groups of eight tokens), the lower one holds the
// address and moves with it, so that one thread issues an MMA in a few
// instructions.  MN-major (tokens are the contraction): `lbo` is the distance
// between 64-element chunks along the head width.
constexpr uint32_t kUmmaDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t umma_lo_kmajor(uint32_t smem_addr) {
    return ((smem_addr >> 4) & 0x3FFFu) | (1u << 16);
}
__device__ __forceinline__ uint32_t umma_lo_mnmajor(uint32_t smem_addr, uint32_t lbo) {
    return ((smem_addr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}

// umma_idesc_f16 with the second operand MN-major.
__host__ __device__ constexpr uint32_t umma_idesc_f16_bmn(bool is_bf16, int M, int N) {
    return umma_idesc_f16(is_bf16, M, N) | (1u << 16);
}

// D[tmem] (+)= A[smem] * B[smem]^T, lower descriptor words.
__device__ __forceinline__ void umma_f16_ss(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(tmem_d),
        "r"(a_lo), "r"(b_lo), "n"(kUmmaDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]: row r of A is lane r, two 16-bit elements of
// the contraction per 32-bit column.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(tmem_d),
        "r"(tmem_a), "r"(b_lo), "n"(kUmmaDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Starts loading 32 consecutive columns of this thread's lane; the values may be
// used after tmem_wait_ld on them.
__device__ __forceinline__ void tmem_start_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Waits for this thread's TMEM loads.  The values pass through, so that no use
// of them can be moved ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    tmem_start_ld_x32(taddr, r);
    tmem_wait_ld(r);
}

// The largest of three (a NaN loses to a number, as with fmaxf).
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Starts storing r[0..31] to 32 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// Starts storing r[0..15] to 16 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two fp32 values rounded to nearest even and packed, `lo` in the low half.
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A TMA view of one (N, L, H, D) operand: a map and factors that are 0 for a
// batch or head axis of stride 0 (it is one entry long in the map).
struct TcView {
    CUtensorMap map;
    int by_n, by_h;
};

// Makes the view of an operand with the given (batch, token, head) strides in
// elements and boxes of `rows` tokens; false when TMA cannot read it (base or
// strides not multiples of 16 bytes, a token stride of 0).  The stride of an
// axis of length 1 does not matter.
inline bool tc_view(TcView *v, const void *base, bool bf16, int N, int L, int H, int D,
                    const int64_t (&stride)[3], int rows) {
    v->by_n = stride[0] == 0 ? 0 : 1;
    v->by_h = stride[2] == 0 ? 0 : 1;
    const uint64_t dims[4] = {(uint64_t)D, v->by_h ? (uint64_t)H : 1, (uint64_t)L,
                              v->by_n ? (uint64_t)N : 1};
    const int64_t by[3] = {stride[2], stride[1], stride[0]};
    uint64_t bytes[3];
    for (int d = 0; d < 3; ++d) {
        bytes[d] = dims[d + 1] == 1 ? 16 : (uint64_t)by[d] * 2;
        if (bytes[d] == 0 || bytes[d] >= (uint64_t(1) << 40)) return false;
    }
    const uint32_t box[4] = {64, 1, (uint32_t)rows, 1};
    return tmap_encode(&v->map, 2, bf16, 4, base, dims, bytes, box, true);
}

// Loads `DP / 64` chunks of ROWS tokens from `row` on, counted in bytes on `bar`.
template <int DP, int ROWS>
__device__ __forceinline__ void tc_load(unsigned char *dst, const TcView &v, int n, int h, int row,
                                        uint64_t *bar) {
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
        tma_load_4d(dst + c * ROWS * 128, &v.map, c * 64, h * v.by_h, row, n * v.by_n, bar);
}

// Scores: D[128 x 64] = A[128 x D] B[64 x D]^T over `steps` steps of 16, at most
// DP / 16; a and b are the tiles' lower descriptor words.
template <int DP>
__device__ __forceinline__ void tc_scores(uint32_t tmem_d, uint32_t a, uint32_t b, uint32_t idesc,
                                          int steps) {
#pragma unroll
    for (int k = 0; k < DP / 16; ++k)
        if (k < steps)   // a step is 32 bytes along a row, four fill a chunk
            umma_f16_ss(tmem_d, a + (k / 4 * kTcM * 128 + k % 4 * 32) / 16,
                        b + (k / 4 * kTcN * 128 + k % 4 * 32) / 16, idesc, k > 0);
}

// Weighted sums: D[128 x width] (+)= A[tmem, 128 x 64] B[64 x width].  The
// 16-bit A lies where the softmax threads read its scores: 16 columns for the
// first 32 tokens, and 16 from column 32 on for the others.
__device__ __forceinline__ void tc_weighted(uint32_t tmem_d, uint32_t tmem_a, uint32_t b,
                                            uint32_t idesc, bool accumulate) {
#pragma unroll
    for (int k = 0; k < kTcN / 16; ++k)
        umma_f16_ts(tmem_d, tmem_a + k / 2 * kTcHalf + k % 2 * 8, b + k * 2048 / 16, idesc,
                    accumulate || k > 0);
}

// Clears token rows [from, ROWS) of a tile (a whole warp calls it): masked
// keys may hold NaN, which a weight of zero would not silence.
template <int DP, int ROWS>
__device__ __forceinline__ void tc_clear_rows(unsigned char *tile, int from) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
        for (int i = from * 8 + lane; i < ROWS * 8; i += 32)
            *reinterpret_cast<uint4 *>(tile + c * ROWS * 128 + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// How a kernel reads the expanded bias: 0 none, 1 a window of it that is copied
// to shared memory with every column tile, 2 global memory.
enum { kBiasNone = 0, kBiasWindow = 1, kBiasGlobal = 2 };

// The window of a column tile: the relative indices of 128 rows against 64
// columns are contiguous, `count` floats from `lowest` (rounded down to 16
// bytes) on, so one bulk copy brings them.  The columns of a one-row grid, or
// of one whose rows are multiples of eight tokens, sit at consecutive indices
// eight at a time (`runs`).
struct TcBias {
    const float *base;   // entry of relative index 0 of head 0; `pad` floats before and after
    int stride;          // floats per head
    int count;           // floats of a window, a multiple of 4
    int below;           // relative indices from the first row and column down to the lowest
    int runs;
};
constexpr int kBiasMost = 2560;   // floats of the largest window that is copied (10 KB)

// First float of the window whose first row and column meet at index r.
__device__ __forceinline__ int bias_start(const TcBias &b, int r) {
    return (r - b.below) & ~3;   // rounds down below zero too
}

// Walks the columns' grid (rows of W tokens, a new row costs P - W more) a tile
// of 64 tokens at a time without dividing: x is the first token's place in its
// row, rel its offset from token 0.  A one-row grid never wraps, also past its
// last token.
struct TileWalk {
    int W, P, x, rel, dy, dx, dy_half, dx_half;
    // Starts at the tile of token `token`.
    __device__ __forceinline__ void init(int rows, int width, int P_, int token = 0) {
        W = rows == 1 ? INT_MAX : width;
        P = rows == 1 ? 0 : P_;
        x = token % W;
        rel = token / W * P + x;
        dy = kTcN / W;
        dx = kTcN - dy * W;
        dy_half = kTcHalf / W;
        dx_half = kTcHalf - dy_half * W;
    }
    __device__ __forceinline__ void next() {
        x += dx;
        rel += dy * P + dx;
        if (x >= W) {
            x -= W;
            rel += P - W;
        }
    }
    // Offset of the tile's token c < 64 from its first one.  `inverse` is
    // 65536 / W + 1, which divides numbers below 128 by W < 64.
    __device__ __forceinline__ int offset(int c, int inverse) const {
        const int at = x + c, rows = W >= kTcN ? at >= W : (at * inverse) >> 16;
        return c + rows * (P - W);
    }
    // Place in its row of the tile's token `part` * 32, and its offset from the
    // tile's first one.
    __device__ __forceinline__ void half(int part, int &x_half, int &rel_half) const {
        x_half = x;
        rel_half = 0;
        if (part) {
            x_half += dx_half;
            rel_half = dy_half * P + dx_half;
            if (x_half >= W) {
                x_half -= W;
                rel_half += P - W;
            }
        }
    }
};

// Offsets of 32 consecutive columns from the first of their tile into a warp's
// 32 ints; columns from `live` of the tile on repeat the last live one.
__device__ __forceinline__ void bias_offsets(int *rel, const TileWalk &walk, int first, int live,
                                             int inverse) {
    const int lane = threadIdx.x % 32;
    __syncwarp();
    rel[lane] = walk.offset(min(first + lane, live - 1), inverse);
    __syncwarp();
}

// The bias of 32 columns of a row.  Column c sits SIGN * (its offset) from `row`
// (SIGN -1: the thread holds a query, columns are keys; +1: a key against
// queries); x and rel as from TileWalk::half.
template <int SIGN>
__device__ __forceinline__ void bias_by_runs(const float *row, int x, int rel, const TileWalk &walk,
                                             float (&b)[kTcHalf]) {
    const int W = walk.W, wrap = walk.P - walk.W;
    if (x + kTcHalf <= W) {   // all in one grid row
        const float *at = row + SIGN * rel;
#pragma unroll
        for (int c = 0; c < kTcHalf; ++c) b[c] = at[SIGN * c];
        return;
    }
#pragma unroll
    for (int c = 0; c < kTcHalf; c += 8) {
        const float *at = row + SIGN * rel;
#pragma unroll
        for (int k = 0; k < 8; ++k) b[c + k] = at[SIGN * k];
        x += 8;
        rel += 8 + (x == W ? wrap : 0);
        x = x == W ? 0 : x;
    }
}
template <int SIGN>
__device__ __forceinline__ void bias_by_table(const float *row, const int *rel,
                                              float (&b)[kTcHalf]) {
#pragma unroll
    for (int c = 0; c < kTcHalf; c += 4) {
        const int4 o = *reinterpret_cast<const int4 *>(rel + c);
        b[c] = row[SIGN * o.x];
        b[c + 1] = row[SIGN * o.y];
        b[c + 2] = row[SIGN * o.z];
        b[c + 3] = row[SIGN * o.w];
    }
}

// r = r * scale + b, on pairs.
__device__ __forceinline__ void scale_and_bias(uint32_t (&r)[kTcHalf], float scale,
                                               const float (&b)[kTcHalf]) {
    const float2 s = make_float2(scale, scale);
#pragma unroll
    for (int c = 0; c < kTcHalf; c += 2) {
        const float2 v = fma_f32x2(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), s,
                                   make_float2(b[c], b[c + 1]));
        r[c] = __float_as_uint(v.x);
        r[c + 1] = __float_as_uint(v.y);
    }
}

// Indices that 64 columns of a grid may span when they are counted past its
// last token as well.
inline int64_t bias_column_span(int rows, int W, int P) {
    return kTcN - 1 + (rows == 1 ? 0 : ((kTcN - 2) / W + 1) * (int64_t)(P - W));
}

// Window of the kernels whose rows are queries, or keys (`by_key`); count 0
// when it is larger than kBiasMost.
inline TcBias tc_bias_of(const AttnArgs &a, bool by_key) {
    TcBias b = {};
    const int64_t rows = by_key ? rel_span(kTcM, a.Lk, a.Hk, a.Wk, a.P)
                                : rel_span(kTcM, a.Lq, a.Hq, a.Wq, a.P);
    const int64_t cols = by_key ? bias_column_span(a.Hq, a.Wq, a.P) : bias_column_span(a.Hk, a.Wk, a.P);
    const int64_t count = (rows + cols + 1 + 3 + 3) / 4 * 4;
    b.below = (int)std::min<int64_t>(by_key ? rows : cols, kBiasMost);
    b.count = count <= kBiasMost ? (int)count : 0;
    b.runs = by_key ? a.Hq == 1 || a.Wq % 8 == 0 : a.Hk == 1 || a.Wk % 8 == 0;
    return b;
}
// Floats kept on both sides of a head's bias: windows reach past its ends.
inline int tc_bias_pad(const AttnArgs &a) {
    return (std::max(tc_bias_of(a, false).count, tc_bias_of(a, true).count) + 8 + 3) / 4 * 4;
}

// Dynamic shared memory of one CTA per SM, at most (barriers, offsets and maxima
// take up to 4 KB of the 227).
constexpr int kTcSmemOne = 223 * 1024;

}  // namespace gs
