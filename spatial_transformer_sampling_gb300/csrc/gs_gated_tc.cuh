// gs_gated_tc.cuh -- the products of the gated projections on the fifth-generation
// tensor cores: a persistent kernel for the forward pass and one for dX, dWg and dWu.
//
// A pair of CTAs (a cluster of two, cta_group::2) works on tiles of 256 rows x NT
// columns.  Each CTA stages its 128 rows of A and NT / 2 rows of B, 64 steps of the
// contraction at a time, by TMA with the 128-byte swizzle; one thread of the pair
// issues tcgen05.mma over both halves, and each CTA's tensor memory receives its 128
// rows.  TMEM holds two tiles, so that the epilogue warps store one while the next is
// multiplied.
//
//   forward  A = X, B = NT / 2 rows of Wg (first CTA) and the same of Wu (second): a
//            tile's columns are G and U of the same NT / 2 outputs, side by side.
//   dX       A = dG, then dU; B = Wg, then Wu, N-major (their rows are contraction).
//   dW       A = dG or dU, M-major; B = X, N-major; the contraction runs over rows.
//
// The tiles of dX and of dWg, dWu are worked on in one launch, the longer contraction
// first and the others where a pair is free (16384 x 1024 x 4096 bf16: 285 us, and 322 in
// two launches of 3.4 and 1.7 tiles per pair).
//
// Bound by the tensor pipe from a contraction of 512 on: forward 16384 x 1024 x 4096
// bf16 in 140 us, 1.96 PFLOP/s, and 173 us with G and U kept, whose 268 MB are written
// meanwhile; backward 285 us, 1.93 PFLOP/s.  Short contractions are bound by the writes:
// 262144 x 64 x 256, kept, 403 MB in 87 us (a fill of that size takes 108).
//
// Both operands are read where they lie: K-major or MN-major is a bit of the
// instruction, nothing is transposed in memory.
//
// Where there are few tiles, a long contraction is shared out: each part's fp32 sums go
// to the workspace and a second kernel adds them in order (262144 rows, D = F = 64
// fp16: 111 us, and a millisecond by the two pairs that dWg and dWu have tiles for).
//
// fp32 operands come as three bf16 planes, x = x0 + x1 + x2 to 2^-24 of x or better,
// and a product is the sum of six of theirs, the small ones first: x2 y0, x0 y2, x1 y1,
// x1 y0, x0 y1, x0 y0 (the other three are below 2^-26 of it).
//
// The tensor cores cut each sum off at the accumulator's last bit: over n steps of
// sixteen products a result is off by up to n 2^-24 of its size, always towards 0.  In
// fp32 the contraction is cut into runs of 4 stages of six products, each accumulated in
// TMEM by itself and added up in the epilogue's registers, rounded to nearest (2.4e-7 of
// the result at D = 2048, the root of the mean square); in 16-bit types no sum in TMEM is
// longer than 512 stages, 1.2e-4 of the result, a quarter of fp16's half step.
#pragma once

#include "gs_attn_tc.cuh"
#include "gs_gated_grad.cuh"

namespace gs {

constexpr int kGtTile = 256;          // rows of a pair's tile
constexpr int kGtHalf = 128;          // rows of A of one CTA
constexpr int kGtK = 64;              // contraction steps per stage: 128 bytes
constexpr int kGtA = kGtHalf * kGtK * 2;   // bytes of A's stage
constexpr int kGtChunk = 64 * kGtK * 2;    // bytes of 64 rows of an MN-major operand
constexpr int kGtSmem = 224 * 1024;
constexpr int kGtRun = 4;             // stages of each product in a run (fp32)
constexpr int kGtLongest = 512;       // stages of a sum in TMEM (16-bit types)

enum { kGtForward = 0, kGtForwardKeep = 1, kGtBackward = 2 };
enum { kGtDx = 0, kGtDw = 1 };   // kinds of a backward tile

// T: type of the outputs.  An epilogue warp has 32 rows and kCols columns of a tile
// (forward: as many of G as of U), which it stages for its stores in boxes of 32 rows:
// sixteen warps of 64 columns in 16-bit types, where what waits for TMEM, the staging
// and the stores is hidden by the other warps (eight warps of 128: 157 us and not 94
// for 262144 x 64 x 256, kept); eight warps of 128 in fp32, whose sums stay in registers.
template <typename T, int MODE, int NT> struct GtShape {
    static constexpr bool kForward = MODE == kGtForward || MODE == kGtForwardKeep;
    static constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
    static constexpr int kCols = sizeof(T) == 4 ? 128 : 64;
    static constexpr int kParts = NT / kCols;        // epilogue warps that share 32 rows
    static constexpr int kEpilogueWarps = 4 * kParts;
    static constexpr int kMmaWarp = kEpilogueWarps, kCopyWarp = kMmaWarp + 1;
    static constexpr int kThreads = (kEpilogueWarps + 2) * 32;
    static constexpr int kB = NT / 2 * kGtK * 2;     // bytes of B's stage
    static constexpr int kStage = kGtA + kB;
    static constexpr int kBoxRow = sizeof(T) == 2 && kForward ? 64 : 128;   // bytes
    static constexpr int kBox = 32 * kBoxRow;
    static constexpr int kBoxCols = kBoxRow / (int)sizeof(T);
    static constexpr int kBoxes = MODE == kGtForwardKeep ? 3 : kForward ? 1 : sizeof(T) == 4 ? 2 : 1;
    static constexpr int kBoxBytes = kBoxes * kEpilogueWarps * kBox;
    static constexpr int kStages = (kGtSmem - kBoxBytes) / kStage < 8 ? (kGtSmem - kBoxBytes) / kStage : 8;
    static constexpr int kSmem = kStages * kStage + kBoxBytes + 1024;
};

// ------------------------------------------------------------------ pairs of CTAs

// The address of this CTA's shared-memory address in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t smem_of_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on a barrier of another CTA of the cluster.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// tc_wait for arrivals from other CTAs.
__device__ __forceinline__ bool tc_wait_cluster(uint64_t *bar, uint32_t parity, unsigned *err) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t n = 1; !mbar_try_wait_cluster(bar, parity); ++n) {
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

// One thread of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, e;\n\t}"
        : "=r"(p));
    return p != 0;
}
// tc_wait by a whole warp.
__device__ __forceinline__ bool gt_wait(uint64_t *bar, uint32_t parity, unsigned *err) {
    return __all_sync(0xffffffffu, tc_wait(bar, parity, err));
}

// Loads a box of a 2-D map into this CTA; its bytes are counted on a barrier of the
// pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1,
                                                 uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(cluster_bar)
        : "memory");
}
// Stores a box from shared memory; what lies outside the tensor is not written.  The
// outputs are the first to leave L2, where the operands are read again: 191 us instead
// of 197 for 16384 x 1024 x 4096, kept.
__device__ __forceinline__ uint64_t first_to_leave() {
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int c0, int c1, uint32_t src,
                                             uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2}], "
        "[%3], %4;" ::"l"(reinterpret_cast<uint64_t>(map)),
        "r"(c0), "r"(c1), "r"(src), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until this thread's bulk stores have read their shared memory.
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(dst))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
// D[tmem of both] (+)= A[smem of both] * B[smem of both]^T, lower descriptor words.
__device__ __forceinline__ void umma_f16_pair(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(tmem_d),
        "r"(a_lo), "r"(b_lo), "n"(kUmmaDescHi), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives on the barrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .b16 both;\n\t"
        "mov.b16 both, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], both;\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

// ------------------------------------------------------------------ arguments

// A 16-bit matrix (rows, width) with rows `pitch` elements apart; planes of fp32 follow
// one another, rows * pitch elements apart.
struct GtMatrix {
    const void *at;
    int64_t rows;
    int width;
    int64_t pitch;
};
constexpr int kGtMostPlanes = 3;

// An output (rows, width): TMA boxes where its rows are multiples of 16 bytes, plain
// stores elsewhere.
struct GtOutput {
    CUtensorMap map;
    void *at;
    int64_t rows;
    int width, boxes;
};

// Tiles of one kind: planes of each operand (forward: a[0], b = Wg and Wu; dX: dG, Wg and
// dU, Wu; dW: dG and dU, b[0]), tiles of 256 rows and NT columns (forward: NT / 2
// outputs), stages of one pair of operands' contraction.
struct GtKind {
    CUtensorMap a[2][kGtMostPlanes], b[2][kGtMostPlanes];
    int tiles_m, tiles_n, k_steps;
    uint32_t per_tiles, per_group;   // 2^32 over the kind's tiles, and over a group's
    // parts of the contraction, and where their sums go: rows of `pitch` floats, a part
    // every `part_stride` floats (backward)
    int parts, pitch;
    float *sums;
    int64_t part_stride;
};

// Which tiles a pair works on: those of kind `first` go round, `turns` and one more for
// the first `extra` pairs; then these take `long_turns` of the other kind's tiles each,
// and the others `short_turns`.
struct GtSchedule {
    int first, turns, extra, long_turns, short_turns, others;
};

struct GtArgs {
    GtKind kind[2];               // forward: the first alone
    GtSchedule plan;
    GtOutput out[3];              // forward: H, G, U; backward: dX, dWg, dWu
    const void *bg, *bu;
    int F;
    ActNumbers act;
    const uint32_t *bound;        // backward in fp16: what dG and dU are scaled by
    unsigned *err;
};

inline bool gt_map(CUtensorMap *map, const GtMatrix &m, bool bf16, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)m.width, (uint64_t)m.rows};
    const uint64_t stride[1] = {m.rows == 1 ? 16 : (uint64_t)m.pitch * 2};
    const uint32_t box[2] = {64, (uint32_t)box_rows};
    return tmap_encode(map, 2, bf16, 2, m.at, dims, stride, box, true);
}
template <typename T>
bool gt_maps(CUtensorMap (&map)[kGtMostPlanes], const GtMatrix &m, int box_rows) {
    constexpr int planes = sizeof(T) == 4 ? 3 : 1;
    for (int i = 0; i < planes; ++i)
        if (!gt_map(&map[i], {(const char *)m.at + i * m.rows * m.pitch * 2, m.rows, m.width, m.pitch},
                    !__is_same(T, __half), box_rows))
            return false;
    return true;
}
template <typename T>
void gt_output(GtOutput *o, void *at, int64_t rows, int width, int box_row) {
    o->at = at;
    o->rows = rows;
    o->width = width;
    const uint64_t dims[2] = {(uint64_t)width, (uint64_t)rows}, stride[1] = {width * sizeof(T)};
    const uint32_t box[2] = {box_row / (uint32_t)sizeof(T), 32};
    o->boxes = width * sizeof(T) % 16 == 0 &&
               tmap_encode(&o->map, sizeof(T), __is_same(T, __nv_bfloat16), 2, at, dims, stride, box,
                           box_row == 128, box_row == 64);
}

// n / d and its remainder by 2^32 / d, rounded down: the estimate is 1 too small at most.
// (Every warp asks for its next tile: by the compiler's division that took 800 cycles, a
// seventh of a tile of 64 channels.)
constexpr uint32_t gt_per(int64_t d) { return d > 1 ? (uint32_t)((int64_t(1) << 32) / d) : 0xFFFFFFFFu; }
__device__ __forceinline__ int gt_divide(int n, int d, uint32_t per, int &rest) {
    int q = (int)__umulhi((uint32_t)n, per);
    rest = n - q * d;
    if (rest >= d) {
        ++q;
        rest -= d;
    }
    return q;
}

// Rows of tiles that are numbered together.
constexpr int kGtGroup = 8;

// The i-th tile of pair `pair` of `pairs`; false when there are no more.  Tiles of a kind
// are numbered eight rows of them at a time, so that those in flight share their operands
// in L2.
struct GtTile {
    int kind, m, n, part;
};
__device__ __forceinline__ bool gt_tile(const GtArgs &p, int pair, int pairs, int i, GtTile &w) {
    const GtSchedule &s = p.plan;
    const bool extra = pair < s.extra;
    const int turns = s.turns + extra;
    int t;
    if (i < turns) {
        w.kind = s.first;
        t = pair + i * pairs;
    } else {
        i -= turns;
        if (i >= (extra ? s.long_turns : s.short_turns)) return false;
        w.kind = 1 - s.first;
        t = extra ? pair + i * s.extra
                  : s.extra * s.long_turns + pair - s.extra + i * (pairs - s.extra);
        if (t >= s.others) return false;
    }
    const GtKind &k = p.kind[w.kind];
    // the parts of all tiles in turn: those in flight read the same rows
    w.part = 0;
    if (k.parts > 1) w.part = gt_divide(t, k.tiles_m * k.tiles_n, k.per_tiles, t);
    int r;
    const int g = gt_divide(t, kGtGroup * k.tiles_n, k.per_group, r);
    const int rows = k.tiles_m - g * kGtGroup;
    if (rows >= kGtGroup) {
        w.m = g * kGtGroup + r % kGtGroup;
        w.n = r / kGtGroup;
    } else {   // the last group, lower than the others
        w.m = g * kGtGroup + r % rows;
        w.n = r / rows;
    }
    return true;
}

// ------------------------------------------------------------------ kernel

// A place in the ring of stages: its parity is that of the phase in which the stage is
// filled for the current turn.
template <int NS> struct GtRing {
    int stage = 0, filled = 0;   // filled: stages passed, NS at most
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        filled += filled < NS;
        if (++stage == NS) {
            stage = 0;
            parity ^= 1;
        }
    }
    __device__ __forceinline__ void back() {
        if (stage-- == 0) {
            stage = NS - 1;
            parity ^= 1;
        }
    }
};

// The products of planes that make up one of fp32 operands, the small ones first.
__device__ __forceinline__ int gt_plane_a(int product) { return (0x201100 >> (20 - 4 * product)) & 3; }
__device__ __forceinline__ int gt_plane_b(int product) { return (0x021010 >> (20 - 4 * product)) & 3; }

// The runs of a tile's contraction (of its part of it) that TMEM accumulates by
// themselves, and a run's stages in order: f(pair of operands, planes of A and B, stage of
// the contraction) until it is false.
struct GtRuns {
    int k_steps, from, to;   // the contraction's stages (fp32: runs) from..to - 1
    template <int PLANES> __device__ __forceinline__ int count() const { return PLANES == 1 ? 1 : to - from; }
};
template <int MODE, int PLANES>
__device__ __forceinline__ GtRuns gt_runs(const GtKind &k, const GtTile &w) {
    const int operands = MODE == kGtBackward && w.kind == kGtDx ? 2 : 1;
    const int all = operands * (PLANES == 1 ? k.k_steps : (k.k_steps + kGtRun - 1) / kGtRun);
    GtRuns r = {k.k_steps, 0, all};
    if (MODE == kGtBackward && k.parts > 1) {
        r.from = (int)((int64_t)all * w.part / k.parts);
        r.to = (int)((int64_t)all * (w.part + 1) / k.parts);
    }
    return r;
}
template <int PLANES, typename F>
__device__ __forceinline__ void gt_steps(const GtRuns &r, int run, F &&f) {
    if (PLANES == 1) {
        for (int k = r.from; k < r.to; ++k) {
            const int which = k >= r.k_steps;
            if (!f(which, 0, 0, k - which * r.k_steps)) return;
        }
        return;
    }
    const int runs = (r.k_steps + kGtRun - 1) / kGtRun, at = r.from + run, which = at >= runs;
    const int k0 = (at - which * runs) * kGtRun, k1 = min(k0 + kGtRun, r.k_steps);
    for (int product = 0; product < 6; ++product)
        for (int k = k0; k < k1; ++k)
            if (!f(which, gt_plane_a(product), gt_plane_b(product), k)) return;
}

// Where 16-byte chunk c of a box's row lies: swizzled as TMA reads it.
template <int ROW> __device__ __forceinline__ int gt_chunk(int row, int c) {
    return row * ROW + (c ^ (ROW == 128 ? row % 8 : row / 2 % 4)) * 16;
}

// A box's staged columns of 32 rows from shared memory to where TMA cannot store.
template <typename T, int ROW>
__device__ __forceinline__ void gt_store_plain(const GtOutput &o, const unsigned char *box,
                                               int64_t row0, int col0) {
    constexpr int N = 4 / (int)sizeof(T), kLanes = ROW / 4;   // columns of a lane, lanes of a row
    const int lane = threadIdx.x % 32, at = lane % kLanes, col = col0 + at * N;
    for (int r = lane / kLanes; r < 32 && row0 + r < o.rows; r += 32 / kLanes) {
        const T *from = reinterpret_cast<const T *>(box + gt_chunk<ROW>(r, at / 4) + at % 4 * 4);
        T *to = (T *)o.at + (row0 + r) * o.width + col;
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (col + e < o.width) to[e] = from[e];
    }
}

// N boxes of a warp, one for each output, all of them at row0 and col0: a lane each.
template <typename T, int ROW, int N>
__device__ __forceinline__ void gt_store_boxes(const GtOutput *out, const unsigned char *box,
                                               int64_t row0, int col0, uint64_t policy) {
    const int lane = threadIdx.x % 32;
    fence_proxy_async_smem();   // all lanes' writes, before the TMA reads them
    __syncwarp();
    if (row0 >= out->rows || col0 >= out->width) return;
    if (lane < N && out[lane].boxes)
        tma_store_2d(&out[lane].map, col0, (int)row0, smem_u32(box + lane * 32 * ROW), policy);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (!out[i].boxes) gt_store_plain<T, ROW>(out[i], box + i * 32 * ROW, row0, col0);
}
// Until a warp's boxes may be written again.
__device__ __forceinline__ void gt_boxes_free() {
    if (threadIdx.x % 32 < 3) {   // the lanes that store
        bulk_commit();
        bulk_wait_read();
    }
    __syncwarp();
}

// N columns of this lane's row into its box from column `col` on, rounded.
template <typename T, int ROW, int N>
__device__ __forceinline__ void gt_stage(unsigned char *box, int col, const float (&v)[N]) {
    const int lane = threadIdx.x % 32;
    constexpr int V = kVec<T>;
#pragma unroll
    for (int i = 0; i < N / V; ++i) {
        uint4 w;
        uint32_t *u = &w.x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 4)
                u[e] = __float_as_uint(v[i * V + e]);
            else
                u[e] = pack2<T>(v[i * V + 2 * e], v[i * V + 2 * e + 1]);
        }
        *reinterpret_cast<uint4 *>(box + gt_chunk<ROW>(lane, col / V + i)) = w;
    }
}

// Loads twice 32 columns of this lane's row from TMEM.
__device__ __forceinline__ void gt_columns_of(uint32_t a, uint32_t b, float (&v)[32], float (&w)[32]) {
    tmem_start_ld_x32(a, reinterpret_cast<uint32_t (&)[32]>(v));
    tmem_start_ld_x32(b, reinterpret_cast<uint32_t (&)[32]>(w));
    tmem_wait_ld(reinterpret_cast<uint32_t (&)[32]>(v));
    tmem_wait_ld(reinterpret_cast<uint32_t (&)[32]>(w));
}

// v += 16 columns of this lane's row in TMEM.
__device__ __forceinline__ void gt_add_columns(uint32_t at, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
#pragma unroll
    for (int c = 0; c < 16; ++c) v[c] += __uint_as_float(r[c]);
}

// v += 32 values that lane i holds the i-th of, by way of 128 bytes of the warp's own.
__device__ __forceinline__ void gt_add_lanes(float (&v)[32], const float *shared) {
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
        const float4 b = *reinterpret_cast<const float4 *>(shared + c);
        v[c] += b.x;
        v[c + 1] += b.y;
        v[c + 2] += b.z;
        v[c + 3] += b.w;
    }
}

template <typename T, int MODE, int NT>
__global__ void __launch_bounds__(GtShape<T, MODE, NT>::kThreads, 1)
    gated_tc_kernel(const __grid_constant__ GtArgs p) {
    using Sh = GtShape<T, MODE, NT>;
    constexpr bool kForward = Sh::kForward;
    constexpr int NS = Sh::kStages, kPlanes = Sh::kPlanes, kRow = Sh::kBoxRow;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], tile_full[2], tile_empty[2], drained;
    __shared__ uint32_t tmem_base;
    unsigned char *stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *boxes = stages + NS * Sh::kStage;
    // the same for a whole warp, and known to be: the loops that copy and multiply are run
    // by whole warps, with their numbers in uniform registers, and one thread issues (by a
    // lane's own loop a stage took 640 cycles to issue, which its MMAs need 512 of)
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    GtTile w;

    if (warp == Sh::kCopyWarp) {   // the maps are there when the first copies want them
        // a plane's maps by four lanes: a[0], a[1], b[0], b[1] of a kind, but for those that
        // it does not have
        const int plane = lane / 4 % 3, of = lane % 4, k = lane / 12;
        const bool has = lane < (kForward ? 12 : 24) && plane < kPlanes &&
                         !(kForward && of == 1) && !(k == kGtDw && of == 3);
        if (has) tma_prefetch_map(of < 2 ? &p.kind[k].a[of][plane] : &p.kind[k].b[of - 2][plane]);
        __syncwarp();
    }
    if (warp == Sh::kMmaWarp) {
        if (lane == 0) {
            for (int s = 0; s < NS; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&tile_full[b], 1);
                mbar_init(&tile_empty[b], 2 * Sh::kEpilogueWarps);
            }
            mbar_init(&drained, 1);
            fence_mbar_init();
        }
        __syncwarp();
        tmem_alloc_pair(&tmem_base);
        tcgen05_fence_before_sync();
    }
    __syncthreads();
    cluster_barrier();   // the other CTA's barriers are set up
    tcgen05_fence_after_sync();
    const uint32_t tmem = tmem_base;
    const void *bg = p.bg, *bu = p.bu;
    wait_for_previous_kernel(bg, bu);
    bool ok = true;

    if (warp == Sh::kCopyWarp) {
        // ---------------------------------------------------- copies, one thread of each CTA
        {
            const bool issues = elect_one();
            GtRing<NS> r;
            for (int i = 0; ok && gt_tile(p, pair, pairs, i, w); ++i) {
                const GtKind &kind = p.kind[w.kind];
                const GtRuns runs = gt_runs<MODE, kPlanes>(kind, w);
                for (int u = 0, units = runs.count<kPlanes>(); u < units && ok; ++u)
                    gt_steps<kPlanes>(runs, u, [&](int which, int pa, int pb, int k) {
                        const int s = r.stage;
                        ok = gt_wait(&empty[s], r.parity ^ 1, p.err);
                        if (!ok) return false;
                        r.next();
                        if (!issues) return true;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * Sh::kStage);
                        const uint32_t bar = smem_of_rank(smem_u32(&full[s]), 0);
                        const uint32_t a = smem_u32(stages + s * Sh::kStage), b = a + kGtA;
                        const int kk = k * kGtK;
                        if (kForward) {
                            tma_load_2d_pair(a, &kind.a[0][pa], kk, w.m * kGtTile + rank * kGtHalf, bar);
                            tma_load_2d_pair(b, &kind.b[rank][pb], kk, w.n * (NT / 2), bar);
                        } else {
                            const int col = w.n * NT + rank * (NT / 2);
                            if (w.kind == kGtDx) {
                                tma_load_2d_pair(a, &kind.a[which][pa], kk,
                                                 w.m * kGtTile + rank * kGtHalf, bar);
                            } else {
                                const int half = kind.tiles_m / 2, of = w.m >= half;
                                const int row = (w.m - of * half) * kGtTile + rank * kGtHalf;
                                tma_load_2d_pair(a, &kind.a[of][pa], row, kk, bar);
                                tma_load_2d_pair(a + kGtChunk, &kind.a[of][pa], row + 64, kk, bar);
                            }
#pragma unroll
                            for (int c = 0; c < NT / 128; ++c)
                                tma_load_2d_pair(b + c * kGtChunk, &kind.b[which][pb], col + c * 64, kk,
                                                 bar);
                        }
                        return true;
                    });
            }
            // every copy lands, and every stage is handed back, before either CTA may
            // leave; where a wait gave up, the copies (counted in the first CTA) land
            const int fills = r.filled;
            for (int i = 0; i < fills; ++i) {
                r.back();
                if (ok)
                    ok = gt_wait(&empty[r.stage], r.parity, p.err);
                else if (rank == 0)
                    gt_wait(&full[r.stage], r.parity, p.err);
            }
        }
        __syncwarp();
    } else if (warp == Sh::kMmaWarp) {
        // ---------------------------------------------------- MMAs, one thread of the pair
        if (rank == 0) {
            const bool issues = elect_one();
            constexpr uint32_t idesc_k = umma_idesc_f16(!__is_same(T, __half), kGtTile, NT) |
                                         (kForward ? 0u : 1u << 16);
            constexpr bool kBmn = !kForward;
            const uint32_t base = smem_u32(stages);
            const uint32_t b0 =
                kBmn ? umma_lo_mnmajor(base + kGtA, kGtChunk) : umma_lo_kmajor(base + kGtA);
            GtRing<NS> r;
            int count = 0;
            for (int t = 0; ok && gt_tile(p, pair, pairs, t, w); ++t) {
                const GtKind &kind = p.kind[w.kind];
                const GtRuns runs = gt_runs<MODE, kPlanes>(kind, w);
                // A is M-major for dW: 16 steps of the contraction are 16 rows, not 32 bytes of one
                const bool amn = !kForward && w.kind == kGtDw;
                const uint32_t idesc = idesc_k | (amn ? 1u << 15 : 0u);
                const uint32_t a0 = amn ? umma_lo_mnmajor(base, kGtChunk) : umma_lo_kmajor(base);
                const uint32_t a_step = (amn ? 2048 : 32) / 16;
                for (int u = 0, units = runs.count<kPlanes>(); u < units && ok; ++u, ++count) {
                    const int b = count & 1;
                    if (count >= 2)
                        ok = __all_sync(0xffffffffu,
                                        tc_wait_cluster(&tile_empty[b], (count / 2 - 1) & 1, p.err));
                    uint32_t more = 0;
                    if (!ok) break;
                    gt_steps<kPlanes>(runs, u, [&](int, int, int, int) {
                        const int s = r.stage;
                        ok = gt_wait(&full[s], r.parity, p.err);
                        if (!ok) return false;
                        r.next();
                        tcgen05_fence_after_sync();
                        const uint32_t a = a0 + s * (Sh::kStage / 16), bb = b0 + s * (Sh::kStage / 16);
                        if (issues) {
#pragma unroll
                            for (int i = 0; i < kGtK / 16; ++i)
                                umma_f16_pair(tmem + b * NT, a + i * a_step,
                                              bb + i * (kBmn ? 2048 : 32) / 16, idesc, i > 0 ? 1u : more);
                            umma_commit_pair(&empty[s]);
                        }
                        more = 1;
                        return true;
                    });
                    if (ok && issues) umma_commit_pair(&tile_full[b]);
                }
            }
            if (!ok) {   // a wait gave up: let the MMAs end before TMEM is released
                if (issues) umma_commit_pair(&drained);
                gt_wait(&drained, 0, p.err);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- epilogue
        const int quarter = warp % 4, part = warp / 4;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        unsigned char *box = boxes + warp * Sh::kBoxes * Sh::kBox;
        // where the warp's i-th 32 columns start in TMEM; forward, U's follow G's
        constexpr int kRuns = Sh::kCols / 32, kHalf = kForward ? kRuns / 2 : kRuns;
        const auto column = [&](int i) { return i / kHalf * (NT / 2) + (part * kHalf + i % kHalf) * 32; };
        const uint64_t policy = first_to_leave();
        int count = 0;
        for (int t = 0; ok && gt_tile(p, pair, pairs, t, w); ++t) {
            const GtKind &kind = p.kind[w.kind];
            const int units = gt_runs<MODE, kPlanes>(kind, w).template count<kPlanes>();
            const int64_t row0 = (int64_t)w.m * kGtTile + rank * kGtHalf + quarter * 32;
            const int f0 = w.n * (NT / 2) + part * kHalf * 32;   // forward: the first output
            float bias[kHalf][2] = {};                           // of outputs f0 + 32 i + lane
            if (kForward && bg)
#pragma unroll
                for (int i = 0; i < kHalf; ++i)
                    if (f0 + i * 32 + lane < p.F) {
                        bias[i][0] = IO<T>::ld((const T *)bg + f0 + i * 32 + lane);
                        bias[i][1] = IO<T>::ld((const T *)bu + f0 + i * 32 + lane);
                    }
            // the warp's columns: of one run in TMEM, or the sums of them all
            float v[kRuns][32];
            if (kPlanes > 1)
#pragma unroll
                for (int i = 0; i < kRuns; ++i)
#pragma unroll
                    for (int c = 0; c < 32; ++c) v[i][c] = 0.0f;
            for (int u = 0; u < units; ++u, ++count) {
                const int b = count & 1;
                ok = __all_sync(0xffffffffu, tc_wait(&tile_full[b], (count / 2) & 1, p.err));
                if (!ok) break;
                tcgen05_fence_after_sync();
                const uint32_t at = tmem + b * NT + lanes;
                if constexpr (kPlanes > 1) {
#pragma unroll
                    for (int i = 0; i < kRuns; ++i) {
                        gt_add_columns(at + column(i), v[i]);
                        gt_add_columns(at + column(i) + 16, v[i] + 16);
                    }
                } else {
                    static_assert(kRuns == 2, "both loads before one wait");
                    gt_columns_of(at + column(0), at + column(1), v[0], v[kRuns - 1]);
                }
                // TMEM is read: the run after next may be multiplied
                tcgen05_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_of_rank(smem_u32(&tile_empty[b]), 0));
            }
            if (!ok) break;
            if constexpr (kForward) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    float(&g)[32] = v[i], (&u)[32] = v[kHalf + i];
                    gt_boxes_free();
                    if (bg) {
                        float *shared = reinterpret_cast<float *>(box);
                        shared[lane] = bias[i][0];
                        shared[32 + lane] = bias[i][1];
                        __syncwarp();
                        gt_add_lanes(g, shared);
                        gt_add_lanes(u, shared + 32);
                        __syncwarp();
                    }
                    if (MODE == kGtForwardKeep) {
                        gt_stage<T, kRow>(box + Sh::kBox, 0, g);
                        gt_stage<T, kRow>(box + 2 * Sh::kBox, 0, u);
                    }
                    act_product<T>(p.act, g, u);
                    gt_stage<T, kRow>(box, 0, g);
                    gt_store_boxes<T, kRow, Sh::kBoxes>(p.out, box, row0, f0 + i * 32, policy);
                }
            } else {
                if constexpr (__is_same(T, __half)) {   // dG and dU are scaled
                    const float f = gated_scale(__ldg(p.bound), true);
#pragma unroll
                    for (int i = 0; i < kRuns; ++i)
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[i][c] *= f;
                }
                const int half = kind.tiles_m / 2, which = w.kind == kGtDw && w.m >= half;
                const GtOutput *out = &p.out[w.kind == kGtDw ? 1 + which : 0];
                const int64_t out_row = row0 - (int64_t)which * half * kGtTile;
                const int col0 = w.n * NT + part * Sh::kCols;
                if (kind.parts > 1) {   // this part's sums, for the kernel that adds them
                    float *to = kind.sums + w.part * kind.part_stride +
                                (which * out->rows + out_row + lane) * kind.pitch + col0;
#pragma unroll
                    for (int i = 0; i < kRuns; ++i)   // the pitch is a multiple of 32
                        if (out_row + lane < out->rows && col0 + i * 32 < kind.pitch)
#pragma unroll
                            for (int c = 0; c < 32; c += 4)
                                *reinterpret_cast<float4 *>(to + i * 32 + c) =
                                    make_float4(v[i][c], v[i][c + 1], v[i][c + 2], v[i][c + 3]);
                    __syncwarp();
                    continue;
                }
                // two runs at a time: a box of both, or one each
#pragma unroll
                for (int i = 0; i < kRuns; i += 2) {
                    gt_boxes_free();
                    if constexpr (Sh::kBoxCols == 64) {
                        gt_stage<T, kRow>(box, 0, v[i]);
                        gt_stage<T, kRow>(box, 32, v[i + 1]);
                        gt_store_boxes<T, kRow, 1>(out, box, out_row, col0 + i * 32, policy);
                    } else {
                        gt_stage<T, kRow>(box, 0, v[i]);
                        gt_stage<T, kRow>(box + Sh::kBox, 0, v[i + 1]);
                        gt_store_boxes<T, kRow, 1>(out, box, out_row, col0 + i * 32, policy);
                        gt_store_boxes<T, kRow, 1>(out, box + Sh::kBox, out_row, col0 + i * 32 + 32,
                                                      policy);
                    }
                }
            }
        }
        gt_boxes_free();
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    cluster_barrier();   // the other CTA neither reads this one's memory nor arrives here any more
    if (warp == Sh::kMmaWarp) tmem_dealloc_pair(tmem);
}

// Pairs of CTAs that the device holds at once.
template <typename T, int MODE, int NT> cudaError_t gt_most_pairs(int *pairs) {
    using Sh = GtShape<T, MODE, NT>;
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    const auto kernel = gated_tc_kernel<T, MODE, NT>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kGatedSms);
    cfg.blockDim = dim3(Sh::kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(pairs, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (*pairs < 1) return cudaErrorInvalidConfiguration;
    if (cached) known[dev].store(*pairs, std::memory_order_release);
    return cudaSuccess;
}

// The schedule of n1 tiles of `steps1` stages each and n2 shorter ones of `steps2` over
// `pairs`, and the stages that the longest of them has (`*length`).
inline GtSchedule gt_schedule(int first, int64_t n1, int64_t steps1, int64_t n2, int64_t steps2,
                              int64_t pairs, int64_t *length) {
    GtSchedule s = {first, (int)(n1 / pairs), (int)(n1 % pairs), 0, 0, (int)n2};
    const int64_t many = s.extra, few = pairs - s.extra;   // pairs with one tile more, and the others
    int64_t by_many = (s.turns + 1) * steps1, by_few = s.turns * steps1, left = n2;
    // whole rounds of all pairs first, then whichever group is done earlier
    const int64_t ahead = steps2 > 0 ? (steps1 + steps2 - 1) / steps2 + 1 : 0;
    const int64_t rounds = n2 / pairs > ahead ? n2 / pairs - ahead : 0;
    s.long_turns = s.short_turns = (int)rounds;
    by_many += rounds * steps2;
    by_few += rounds * steps2;
    left -= rounds * pairs;
    while (left > 0) {
        if (many > 0 && by_many + steps2 < by_few + steps2) {
            ++s.long_turns;
            by_many += steps2;
            left -= many;
        } else {
            ++s.short_turns;
            by_few += steps2;
            left -= few;
        }
    }
    *length = many > 0 && by_many > by_few ? by_many : by_few;
    return s;
}

template <typename T, int MODE, int NT>
cudaError_t launch_gt_as(GtArgs &p, bool follows, cudaStream_t s) {
    using Sh = GtShape<T, MODE, NT>;
    int pairs = 0;
    const cudaError_t e = gt_most_pairs<T, MODE, NT>(&pairs);
    if (e != cudaSuccess) return e;
    const auto tiles = [&](int k) { return (int64_t)p.kind[k].tiles_m * p.kind[k].tiles_n * p.kind[k].parts; };
    const auto stages = [&](int k) {   // of a tile's part
        const int64_t all = (int64_t)p.kind[k].k_steps * (MODE == kGtBackward && k == kGtDx ? 2 : 1);
        return p.kind[k].parts ? (all + p.kind[k].parts - 1) / p.kind[k].parts : 0;
    };
    const int64_t n0 = tiles(0), n1 = tiles(1), k0 = stages(0), k1 = stages(1);
    if (n0 + n1 < pairs) pairs = (int)(n0 + n1);
    for (GtKind &k : p.kind) {
        k.per_tiles = gt_per((int64_t)k.tiles_m * k.tiles_n);
        k.per_group = gt_per((int64_t)kGtGroup * k.tiles_n);
    }
    int64_t length;
    p.plan = k0 >= k1 ? gt_schedule(0, n0, k0, n1, k1, pairs, &length)
                      : gt_schedule(1, n1, k1, n0, k0, pairs, &length);
    return launch_next(LaunchAs(follows, 2), gated_tc_kernel<T, MODE, NT>, dim3(2 * pairs),
                       Sh::kThreads, Sh::kSmem, s, p);
}

// What a stage takes in us with tiles of 128 columns (its copies bound it) and of 256
// (its MMAs), as measured.
constexpr double gt_stage_us(int nt) { return nt == 128 ? 0.216 : 0.302; }
constexpr int kGtPairs = kGatedSms / 2;

// How the backward products are laid out: columns of a tile, parts of each kind's
// contraction, and the workspace of the parts' sums.
struct GtBackwardPlan {
    int columns, parts[2], pitch;
    int64_t sums[2];   // floats
    int64_t bytes() const { return (sums[0] + sums[1]) * 4; }
};
template <typename T> GtBackwardPlan gt_backward_plan(const GatedArgs &a) {
    const int products = sizeof(T) == 4 ? 6 : 1;
    const int64_t rows_of[2] = {a.rows, 2 * (int64_t)a.F};
    const int64_t tiles_m[2] = {(a.rows + kGtTile - 1) / kGtTile,
                                2 * (((int64_t)a.F + kGtTile - 1) / kGtTile)};
    const int64_t k[2] = {2 * (((int64_t)a.F + kGtK - 1) / kGtK), (a.rows + kGtK - 1) / kGtK};
    GtBackwardPlan best = {};
    double least = 0.0;
    for (const int nt : {256, 128})
        for (const bool share : {false, true}) {
            GtBackwardPlan q = {nt, {1, 1}, (a.D + 31) / 32 * 32, {0, 0}};
            const int64_t n = (a.D + nt - 1) / nt;
            const int64_t even = (n * (tiles_m[0] * k[0] + tiles_m[1] * k[1]) + kGtPairs - 1) / kGtPairs;
            double us = 0.0;
            // shared out: parts of what a pair has, of eight stages at least
            int64_t most = share ? (even > 8 ? even : 8) : INT64_MAX;
            if (sizeof(T) == 2 && most > kGtLongest) most = kGtLongest;
            for (int i = 0; i < 2; ++i) {
                q.parts[i] = (int)((k[i] - 1) / most) + 1;
                if (q.parts[i] > 1) q.sums[i] = q.parts[i] * rows_of[i] * q.pitch;
            }
            if (q.bytes() > 0) us = 5.0 + 2.0 * (double)q.bytes() / 4e6;   // a kernel more, at 4 TB/s
            const int64_t n0 = n * tiles_m[0] * q.parts[0], n1 = n * tiles_m[1] * q.parts[1];
            const int64_t k0 = (k[0] + q.parts[0] - 1) / q.parts[0], k1 = (k[1] + q.parts[1] - 1) / q.parts[1];
            int64_t length;
            if (k0 >= k1)
                gt_schedule(kGtDx, n0, k0, n1, k1, kGtPairs, &length);
            else
                gt_schedule(kGtDw, n1, k1, n0, k0, kGtPairs, &length);
            us += (double)length * products * gt_stage_us(nt);
            if (best.columns == 0 || us < least) {
                best = q;
                least = us;
            }
        }
    return best;
}

// The sums of the parts, added in order and rounded: four columns a thread.
struct GtJoin {
    const float *from[2];
    int parts[2], pitch, D;
    int64_t rows[2], part_stride[2];   // dX's rows; dWg's and then dWu's
    void *dX, *dWg, *dWu;
};
template <typename T> __global__ void __launch_bounds__(256) gated_join_kernel(GtJoin j) {
    const int kind = blockIdx.y, quads = j.pitch / 4;
    const int parts = kind ? j.parts[1] : j.parts[0];
    const float *from = kind ? j.from[1] : j.from[0];
    const int64_t rows = kind ? j.rows[1] : j.rows[0], stride = kind ? j.part_stride[1] : j.part_stride[0];
    wait_for_previous_kernel(from);
    if (parts < 2) return;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * quads; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / quads;
        const int d = (int)(i - r * quads) * 4;
        if (d >= j.D) continue;
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float4 x = *reinterpret_cast<const float4 *>(from + s * stride + r * j.pitch + d);
            t.x += x.x;
            t.y += x.y;
            t.z += x.z;
            t.w += x.w;
        }
        const int64_t half = rows / 2;
        T *out = kind == kGtDx ? (T *)j.dX + r * j.D
                 : r < half    ? (T *)j.dWg + r * j.D
                               : (T *)j.dWu + (r - half) * j.D;
        const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (d + e < j.D) out[d + e] = IO<T>::st(v[e]);
    }
}

// Whether a forward row's sum in TMEM is not too long.
template <typename T> bool gt_forward_takes(const GatedArgs &a) {
    return sizeof(T) == 4 || a.D <= kGtLongest * kGtK;
}

// Forward pass from 16-bit operands (T float: planes); *used: TMA takes them.
template <typename T>
cudaError_t launch_gt_forward(const GatedArgs &a, const GatedPtrs &q, const GtMatrix &X,
                              const GtMatrix &Wg, const GtMatrix &Wu, bool follows, cudaStream_t s,
                              bool *used) {
    GtArgs p = {};
    GtKind &k = p.kind[0];
    k.tiles_m = (int)((a.rows + kGtTile - 1) / kGtTile);
    k.k_steps = (a.D + kGtK - 1) / kGtK;
    const auto tiles_n = [&](int nt) { return (a.F + nt / 2 - 1) / (nt / 2); };
    const auto us = [&](int nt) {
        return (double)(((int64_t)k.tiles_m * tiles_n(nt) + kGtPairs - 1) / kGtPairs) * gt_stage_us(nt);
    };
    const bool narrow = us(128) < us(256);
    const int nt = narrow ? 128 : 256;
    k.tiles_n = tiles_n(nt);
    k.parts = 1;
    *used = gt_maps<T>(k.a[0], X, kGtHalf) && gt_maps<T>(k.b[0], Wg, nt / 2) &&
            gt_maps<T>(k.b[1], Wu, nt / 2);
    if (!*used) return cudaSuccess;
    const int box_row = GtShape<T, kGtForward, 256>::kBoxRow;
    gt_output<T>(&p.out[0], q.H, a.rows, a.F, box_row);
    if (q.G) {
        gt_output<T>(&p.out[1], q.G, a.rows, a.F, box_row);
        gt_output<T>(&p.out[2], q.U, a.rows, a.F, box_row);
    }
    p.bg = q.bg;
    p.bu = q.bu;
    p.F = a.F;
    p.act = act_numbers(a.act);
    p.err = a.err;
    if (narrow)
        return q.G ? launch_gt_as<T, kGtForwardKeep, 128>(p, follows, s)
                   : launch_gt_as<T, kGtForward, 128>(p, follows, s);
    return q.G ? launch_gt_as<T, kGtForwardKeep, 256>(p, follows, s)
               : launch_gt_as<T, kGtForward, 256>(p, follows, s);
}

// dX, dWg and dWu from 16-bit operands (T float: planes); *used: TMA takes them.
template <typename T>
cudaError_t launch_gt_backward(const GatedArgs &a, const GatedPtrs &q, const GtMatrix &X,
                               const GtMatrix &Wg, const GtMatrix &Wu, const GtMatrix &dG,
                               const GtMatrix &dU, const uint32_t *bound, float *sums, bool follows,
                               cudaStream_t s, bool *used) {
    GtArgs p = {};
    GtKind &x = p.kind[kGtDx], &w = p.kind[kGtDw];
    *used = gt_maps<T>(x.a[0], dG, kGtHalf) && gt_maps<T>(x.a[1], dU, kGtHalf) &&
            gt_maps<T>(x.b[0], Wg, kGtK) && gt_maps<T>(x.b[1], Wu, kGtK) &&
            gt_maps<T>(w.a[0], dG, kGtK) && gt_maps<T>(w.a[1], dU, kGtK) &&
            gt_maps<T>(w.b[0], X, kGtK);
    if (!*used) return cudaSuccess;
    gt_output<T>(&p.out[0], q.dX, a.rows, a.D, 128);
    gt_output<T>(&p.out[1], q.dWg, a.F, a.D, 128);
    gt_output<T>(&p.out[2], q.dWu, a.F, a.D, 128);
    p.err = a.err;
    p.bound = bound;
    x.tiles_m = (int)((a.rows + kGtTile - 1) / kGtTile);
    x.k_steps = (a.F + kGtK - 1) / kGtK;
    w.tiles_m = 2 * ((a.F + kGtTile - 1) / kGtTile);
    w.k_steps = (int)((a.rows + kGtK - 1) / kGtK);
    const GtBackwardPlan plan = gt_backward_plan<T>(a);
    const int nt = plan.columns;
    x.tiles_n = w.tiles_n = (a.D + nt - 1) / nt;
    const int64_t rows_of[2] = {a.rows, 2 * (int64_t)a.F};
    for (int i = 0; i < 2; ++i) {
        p.kind[i].parts = plan.parts[i];
        p.kind[i].pitch = plan.pitch;
        p.kind[i].sums = sums + (i ? plan.sums[0] : 0);
        p.kind[i].part_stride = rows_of[i] * plan.pitch;
    }
    const cudaError_t e = nt == 128 ? launch_gt_as<T, kGtBackward, 128>(p, follows, s)
                                    : launch_gt_as<T, kGtBackward, 256>(p, follows, s);
    if (e != cudaSuccess || plan.bytes() == 0) return e;
    const GtJoin j = {{x.sums, w.sums},     {x.parts, w.parts},
                      plan.pitch,           a.D,
                      {rows_of[0], rows_of[1]}, {x.part_stride, w.part_stride},
                      q.dX,                 q.dWg,
                      q.dWu};
    const int64_t most = (x.parts > 1 && (w.parts < 2 || rows_of[0] > rows_of[1]) ? rows_of[0] : rows_of[1]) *
                         (plan.pitch / 4);
    const int64_t need = (most + 255) / 256;
    return launch_next(true, gated_join_kernel<T>,
                       dim3((unsigned)(need < 8 * kGatedSms ? need : 8 * kGatedSms), 2), 256, 0, s, j);
}

}  // namespace gs
