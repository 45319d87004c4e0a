// gs_gated_tc.cuh -- the products of the gated projections on the fifth-generation
// tensor cores: one persistent kernel for the forward pass, for dX and for dWg, dWu.
//
// A pair of CTAs (a cluster of two, cta_group::2) works on tiles of 256 rows x 256
// columns.  Each CTA stages its 128 rows of A and 128 rows of B, 64 steps of the
// contraction at a time, by TMA with the 128-byte swizzle; one thread of the pair
// issues tcgen05.mma over both halves, and each CTA's tensor memory receives its 128
// rows.  TMEM holds two tiles, so that eight epilogue warps store one while the next
// is multiplied.
//
//   forward  A = X, B = 128 rows of Wg (first CTA) and the same 128 of Wu (second):
//            a tile's columns are G and U of the same 128 outputs, side by side.
//   dX       A = dG, then dU; B = Wg, then Wu, N-major (their rows are contraction).
//   dW       A = dG or dU, M-major; B = X, N-major; the contraction runs over rows.
//
// Both operands are read where they lie: K-major or MN-major is a bit of the
// instruction, nothing is transposed in memory.
#pragma once

#include "gs_attn_tc.cuh"
#include "gs_gated.cuh"

namespace gs {

constexpr int kGtEpilogueWarps = 8;
constexpr int kGtMmaWarp = kGtEpilogueWarps, kGtCopyWarp = kGtMmaWarp + 1;
constexpr int kGtThreads = (kGtEpilogueWarps + 2) * 32;
constexpr int kGtTile = 256;          // rows and columns of a pair's tile
constexpr int kGtHalf = 128;          // rows of A, and of B, of one CTA
constexpr int kGtK = 64;              // contraction steps per stage: 128 bytes
constexpr int kGtOperand = kGtHalf * kGtK * 2;          // bytes of one operand's stage
constexpr int kGtStage = 2 * kGtOperand;
constexpr int kGtBox = 32 * 64 * 2;   // bytes of a warp's staged output box, 32 rows x 64 columns
constexpr int kGtSmem = 224 * 1024;

enum { kGtForward = 0, kGtForwardKeep = 1, kGtDx = 2, kGtDw = 3 };

template <int MODE> struct GtShape {
    static constexpr int kBoxes = MODE == kGtForwardKeep ? 3 : MODE == kGtForward ? 1 : 2;
    static constexpr int kBoxBytes = kBoxes * kGtEpilogueWarps * kGtBox;
    static constexpr int kStages = (kGtSmem - kBoxBytes) / kGtStage;
    static constexpr int kSmem = kStages * kGtStage + kBoxBytes + 1024;
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
// Stores a box from shared memory; what lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, int c0, int c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
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

// A 16-bit matrix (rows, width) with rows `pitch` elements apart.
struct GtMatrix {
    const void *at;
    int64_t rows;
    int width;
    int64_t pitch;
};

// An output (rows, width): TMA boxes where its rows are multiples of 16 bytes, plain
// stores elsewhere.
struct GtOutput {
    CUtensorMap map;
    void *at;
    int64_t rows;
    int width, boxes;
};

struct GtArgs {
    CUtensorMap a[2], b[2];       // forward: a[0], b = Wg and Wu; dX: dG, Wg and dU, Wu; dW: b[0]
    GtOutput out[3];              // forward: H, G, U; dX: dX; dW: dWg, dWu
    const void *bg, *bu;
    int F, act, bias_runs;        // bias_runs: the biases are 16-byte aligned
    int tiles_m, tiles_n;         // of 256 rows, and 256 columns (forward: 128 outputs)
    int k_steps;                  // of one pair of operands
    unsigned *err;
};

inline bool gt_map(CUtensorMap *map, const GtMatrix &m, bool bf16, int box_rows) {
    const uint64_t dims[2] = {(uint64_t)m.width, (uint64_t)m.rows};
    const uint64_t stride[1] = {m.rows == 1 ? 16 : (uint64_t)m.pitch * 2};
    const uint32_t box[2] = {64, (uint32_t)box_rows};
    return tmap_encode(map, 2, bf16, 2, m.at, dims, stride, box, true);
}
inline void gt_output(GtOutput *o, void *at, int64_t rows, int width, bool bf16) {
    o->at = at;
    o->rows = rows;
    o->width = width;
    o->boxes = width % 8 == 0 && gt_map(&o->map, {at, rows, width, width}, bf16, 32);
}

// Tile t of tiles_m x tiles_n: eight rows of tiles at a time, so that the tiles in
// flight share their operands in L2.
struct GtTile {
    int m, n;
};
__device__ __forceinline__ GtTile gt_tile(const GtArgs &p, int t) {
    constexpr int kGroup = 8;
    const int per = kGroup * p.tiles_n, g = t / per, r = t - g * per;
    const int rows = min(kGroup, p.tiles_m - g * kGroup);
    return {g * kGroup + r % rows, r / rows};
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

// 64 staged columns of 32 rows from shared memory to where TMA cannot store.
template <typename T>
__device__ __forceinline__ void gt_store_plain(const GtOutput &o, const unsigned char *box,
                                               int64_t row0, int col0) {
    const int lane = threadIdx.x % 32, c = lane * 2;
    for (int r = 0; r < 32 && row0 + r < o.rows; ++r) {
        const T *from = reinterpret_cast<const T *>(box + r * 128 + (((c / 8) ^ (r % 8)) * 16)) + c % 8;
        T *to = (T *)o.at + (row0 + r) * o.width + col0 + c;
        if (col0 + c < o.width) to[0] = from[0];
        if (col0 + c + 1 < o.width) to[1] = from[1];
    }
}

// A warp's box of 32 rows x 64 columns, written by all its lanes, to the output.
template <typename T>
__device__ __forceinline__ void gt_store_box(const GtOutput &o, const unsigned char *box, int64_t row0,
                                             int col0) {
    if (o.boxes) fence_proxy_async_smem();
    __syncwarp();
    if (row0 >= o.rows || col0 >= o.width) return;
    if (o.boxes) {
        if (threadIdx.x % 32 == 0) tma_store_2d(&o.map, col0, (int)row0, smem_u32(box));
    } else {
        gt_store_plain<T>(o, box, row0, col0);
    }
}

// 32 packed columns (16 words) of this lane's row into its box, chunks from `chunk` on.
__device__ __forceinline__ void gt_stage(unsigned char *box, int chunk, const uint32_t (&w)[16]) {
    const int lane = threadIdx.x % 32;
    unsigned char *row = box + lane * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(row + (((chunk + i) ^ (lane % 8)) * 16)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// v += 32 biases from column f on; the same for all lanes.
template <typename T>
__device__ __forceinline__ void gt_add_bias(uint32_t (&v)[32], const T *bias, int f, int F, bool runs) {
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        float b[8] = {};
        if (runs && f + c + 8 <= F) {
            Run<T, 8>::widen(__ldg(reinterpret_cast<const uint4 *>(bias + f + c)), b);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (f + c + e < F) b[e] = IO<T>::ld(bias + f + c + e);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c + e] = __float_as_uint(__uint_as_float(v[c + e]) + b[e]);
    }
}

template <typename T> __device__ __forceinline__ void gt_pack(const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        w[i] = pack2<T>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kGtThreads, 1) gated_tc_kernel(const __grid_constant__ GtArgs p) {
    using Sh = GtShape<MODE>;
    constexpr bool kForward = MODE == kGtForward || MODE == kGtForwardKeep;
    constexpr bool kBf16 = __is_same(T, __nv_bfloat16);
    constexpr int NS = Sh::kStages;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full[NS], empty[NS], tile_full[2], tile_empty[2], drained;
    __shared__ uint32_t tmem_base;
    unsigned char *stages = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    unsigned char *boxes = stages + NS * kGtStage;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int tiles = p.tiles_m * p.tiles_n;
    const int steps = MODE == kGtDx ? 2 * p.k_steps : p.k_steps;

    if (warp == kGtMmaWarp) {
        if (lane == 0) {
            for (int s = 0; s < NS; ++s) {
                mbar_init(&full[s], 1);
                mbar_init(&empty[s], 1);
            }
            for (int b = 0; b < 2; ++b) {
                mbar_init(&tile_full[b], 1);
                mbar_init(&tile_empty[b], 2 * kGtEpilogueWarps);
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

    if (warp == kGtCopyWarp) {
        // ---------------------------------------------------- copies, one thread of each CTA
        if (lane == 0) {
            GtRing<NS> r;
            for (int t = pair; t < tiles && ok; t += pairs) {
                const GtTile w = gt_tile(p, t);
                for (int k = 0; k < steps; ++k, r.next()) {
                    const int s = r.stage;
                    ok = tc_wait(&empty[s], r.parity ^ 1, p.err);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kGtStage);
                    const uint32_t bar = smem_of_rank(smem_u32(&full[s]), 0);
                    const uint32_t a = smem_u32(stages + s * kGtStage), b = a + kGtOperand;
                    if (kForward) {
                        tma_load_2d_pair(a, &p.a[0], k * kGtK, w.m * kGtTile + rank * kGtHalf, bar);
                        tma_load_2d_pair(b, &p.b[rank], k * kGtK, w.n * kGtHalf, bar);
                    } else if (MODE == kGtDx) {
                        const int which = k >= p.k_steps, kk = (k - which * p.k_steps) * kGtK;
                        const int col = w.n * kGtTile + rank * kGtHalf;
                        tma_load_2d_pair(a, &p.a[which], kk, w.m * kGtTile + rank * kGtHalf, bar);
                        tma_load_2d_pair(b, &p.b[which], col, kk, bar);
                        tma_load_2d_pair(b + kGtOperand / 2, &p.b[which], col + 64, kk, bar);
                    } else {
                        const int half = p.tiles_m / 2, which = w.m >= half;
                        const int row = (w.m - which * half) * kGtTile + rank * kGtHalf;
                        const int col = w.n * kGtTile + rank * kGtHalf;
                        tma_load_2d_pair(a, &p.a[which], row, k * kGtK, bar);
                        tma_load_2d_pair(a + kGtOperand / 2, &p.a[which], row + 64, k * kGtK, bar);
                        tma_load_2d_pair(b, &p.b[0], col, k * kGtK, bar);
                        tma_load_2d_pair(b + kGtOperand / 2, &p.b[0], col + 64, k * kGtK, bar);
                    }
                }
            }
            // every copy lands, and every stage is handed back, before either CTA may
            // leave; where a wait gave up, the copies (counted in the first CTA) land
            const int fills = r.filled < NS ? r.filled : NS;
            for (int i = 0; i < fills; ++i) {
                r.back();
                if (ok)
                    ok = tc_wait(&empty[r.stage], r.parity, p.err);
                else if (rank == 0)
                    tc_wait(&full[r.stage], r.parity, p.err);
            }
        }
        __syncwarp();
    } else if (warp == kGtMmaWarp) {
        // ---------------------------------------------------- MMAs, one thread of the pair
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = umma_idesc_f16(kBf16, kGtTile, kGtTile) |
                                       (MODE == kGtDw ? 1u << 15 : 0u) | (kForward ? 0u : 1u << 16);
            constexpr bool kAmn = MODE == kGtDw, kBmn = !kForward;
            const uint32_t base = smem_u32(stages);
            const uint32_t a0 = kAmn ? umma_lo_mnmajor(base, kGtOperand / 2) : umma_lo_kmajor(base);
            const uint32_t b0 = kBmn ? umma_lo_mnmajor(base + kGtOperand, kGtOperand / 2)
                                     : umma_lo_kmajor(base + kGtOperand);
            GtRing<NS> r;
            int count = 0;
            for (int t = pair; t < tiles && ok; t += pairs, ++count) {
                const int b = count & 1;
                if (count >= 2) ok = tc_wait_cluster(&tile_empty[b], (count / 2 - 1) & 1, p.err);
                for (int k = 0; k < steps && ok; ++k, r.next()) {
                    const int s = r.stage;
                    ok = tc_wait(&full[s], r.parity, p.err);
                    if (!ok) break;
                    tcgen05_fence_after_sync();
                    const uint32_t a = a0 + s * (kGtStage / 16), bb = b0 + s * (kGtStage / 16);
#pragma unroll
                    for (int i = 0; i < kGtK / 16; ++i)   // 16 steps: 32 bytes of a row, or 16 rows
                        umma_f16_pair(tmem + b * kGtTile, a + i * (kAmn ? 2048 : 32) / 16,
                                      bb + i * (kBmn ? 2048 : 32) / 16, idesc, k > 0 || i > 0);
                    umma_commit_pair(&empty[s]);
                }
                if (ok) umma_commit_pair(&tile_full[b]);
            }
            if (!ok) {   // a wait gave up: let the MMAs end before TMEM is released
                umma_commit_pair(&drained);
                tc_wait(&drained, 0, p.err);
            }
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------- epilogue
        const int quarter = warp % 4, part = warp / 4;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        unsigned char *box = boxes + warp * Sh::kBoxes * kGtBox;
        int count = 0;
        for (int t = pair; t < tiles && ok; t += pairs, ++count) {
            const GtTile w = gt_tile(p, t);
            const int b = count & 1;
            ok = __all_sync(0xffffffffu, tc_wait(&tile_full[b], (count / 2) & 1, p.err));
            if (!ok) break;
            tcgen05_fence_after_sync();
            const uint32_t at = tmem + b * kGtTile + lanes;
            const auto release = [&] {   // TMEM is read: the tile after next may be multiplied
                tcgen05_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(smem_of_rank(smem_u32(&tile_empty[b]), 0));
            };
            if (lane == 0) bulk_wait_read();
            __syncwarp();
            const int64_t row0 = (int64_t)w.m * kGtTile + rank * kGtHalf + quarter * 32;
            if constexpr (kForward) {
                const int f0 = w.n * kGtHalf + part * 64;
#pragma unroll 1
                for (int c = 0; c < 64; c += 32) {
                    uint32_t g[32], u[32], h[32], packed[16];
                    tmem_start_ld_x32(at + part * 64 + c, g);
                    tmem_start_ld_x32(at + kGtHalf + part * 64 + c, u);
                    tmem_wait_ld(g);
                    tmem_wait_ld(u);
                    if (c == 32) release();
                    if (bg) {
                        gt_add_bias(g, (const T *)bg, f0 + c, p.F, p.bias_runs);
                        gt_add_bias(u, (const T *)bu, f0 + c, p.F, p.bias_runs);
                    }
                    with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            h[i] = __float_as_uint(act_of<decltype(act)::value>(__uint_as_float(g[i])) *
                                                   __uint_as_float(u[i]));
                    });
                    gt_pack<T>(h, packed);
                    gt_stage(box, c / 8, packed);
                    if (MODE == kGtForwardKeep) {
                        gt_pack<T>(g, packed);
                        gt_stage(box + kGtBox, c / 8, packed);
                        gt_pack<T>(u, packed);
                        gt_stage(box + 2 * kGtBox, c / 8, packed);
                    }
                }
#pragma unroll
                for (int o = 0; o < Sh::kBoxes; ++o)
                    gt_store_box<T>(p.out[o], box + o * kGtBox, row0, f0);
            } else {
                const int half = p.tiles_m / 2, which = MODE == kGtDw && w.m >= half;
                const GtOutput &out = p.out[which];
                const int64_t out_row = row0 - (int64_t)which * half * kGtTile;
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t x[32], y[32], packed[16];
                    tmem_start_ld_x32(at + part * 128 + c, x);
                    tmem_start_ld_x32(at + part * 128 + c + 32, y);
                    tmem_wait_ld(x);
                    tmem_wait_ld(y);
                    if (c == 64) release();
                    unsigned char *to = box + c / 64 * kGtBox;
                    gt_pack<T>(x, packed);
                    gt_stage(to, 0, packed);
                    gt_pack<T>(y, packed);
                    gt_stage(to, 4, packed);
                    gt_store_box<T>(out, to, out_row, w.n * kGtTile + part * 128 + c);
                }
            }
            if (lane == 0) bulk_commit();
            __syncwarp();
        }
        if (lane == 0) bulk_wait_read();
        __syncwarp();
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    cluster_barrier();   // the other CTA neither reads this one's memory nor arrives here any more
    if (warp == kGtMmaWarp) tmem_dealloc_pair(tmem);
}

// Pairs of CTAs that the device holds at once.
template <typename T, int MODE> cudaError_t gt_most_pairs(int *pairs) {
    static std::atomic<int> known[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool cached = dev >= 0 && dev < kMaxDevices;
    if (cached && (*pairs = known[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
    const auto kernel = gated_tc_kernel<T, MODE>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GtShape<MODE>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kGatedSms);
    cfg.blockDim = dim3(kGtThreads);
    cfg.dynamicSmemBytes = GtShape<MODE>::kSmem;
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

template <typename T, int MODE>
cudaError_t launch_gt(const GtArgs &p, bool follows, cudaStream_t s) {
    int pairs = 0;
    const cudaError_t e = gt_most_pairs<T, MODE>(&pairs);
    if (e != cudaSuccess) return e;
    const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
    const unsigned blocks = 2 * (unsigned)(tiles < pairs ? tiles : pairs);
    return launch_next(LaunchAs(follows, 2), gated_tc_kernel<T, MODE>, dim3(blocks), kGtThreads,
                       GtShape<MODE>::kSmem, s, p);
}

// Forward pass from 16-bit operands; *used: TMA takes them.
template <typename T>
cudaError_t launch_gt_forward(const GatedArgs &a, const GatedPtrs &q, const GtMatrix &X,
                              const GtMatrix &Wg, const GtMatrix &Wu, bool follows, cudaStream_t s,
                              bool *used) {
    constexpr bool bf16 = __is_same(T, __nv_bfloat16);
    GtArgs p = {};
    *used = gt_map(&p.a[0], X, bf16, kGtHalf) && gt_map(&p.b[0], Wg, bf16, kGtHalf) &&
            gt_map(&p.b[1], Wu, bf16, kGtHalf);
    if (!*used) return cudaSuccess;
    gt_output(&p.out[0], q.H, a.rows, a.F, bf16);
    if (q.G) {
        gt_output(&p.out[1], q.G, a.rows, a.F, bf16);
        gt_output(&p.out[2], q.U, a.rows, a.F, bf16);
    }
    p.bg = q.bg;
    p.bu = q.bu;
    p.bias_runs = aligned16(q.bg) && aligned16(q.bu);
    p.F = a.F;
    p.act = a.act;
    p.tiles_m = (int)((a.rows + kGtTile - 1) / kGtTile);
    p.tiles_n = (a.F + kGtHalf - 1) / kGtHalf;
    p.k_steps = (a.D + kGtK - 1) / kGtK;
    p.err = a.err;
    return q.G ? launch_gt<T, kGtForwardKeep>(p, follows, s) : launch_gt<T, kGtForward>(p, follows, s);
}

// dX, dWg and dWu from 16-bit operands; *used: TMA takes them.
template <typename T>
cudaError_t launch_gt_backward(const GatedArgs &a, const GatedPtrs &q, const GtMatrix &X,
                               const GtMatrix &Wg, const GtMatrix &Wu, const GtMatrix &dG,
                               const GtMatrix &dU, bool follows, cudaStream_t s, bool *used) {
    constexpr bool bf16 = __is_same(T, __nv_bfloat16);
    GtArgs x = {}, w = {};
    *used = gt_map(&x.a[0], dG, bf16, kGtHalf) && gt_map(&x.a[1], dU, bf16, kGtHalf) &&
            gt_map(&x.b[0], Wg, bf16, kGtK) && gt_map(&x.b[1], Wu, bf16, kGtK) &&
            gt_map(&w.a[0], dG, bf16, kGtK) && gt_map(&w.a[1], dU, bf16, kGtK) &&
            gt_map(&w.b[0], X, bf16, kGtK);
    if (!*used) return cudaSuccess;
    gt_output(&x.out[0], q.dX, a.rows, a.D, bf16);
    x.tiles_m = (int)((a.rows + kGtTile - 1) / kGtTile);
    x.tiles_n = (a.D + kGtTile - 1) / kGtTile;
    x.k_steps = (a.F + kGtK - 1) / kGtK;
    x.err = a.err;
    gt_output(&w.out[0], q.dWg, a.F, a.D, bf16);
    gt_output(&w.out[1], q.dWu, a.F, a.D, bf16);
    w.tiles_m = 2 * ((a.F + kGtTile - 1) / kGtTile);
    w.tiles_n = (a.D + kGtTile - 1) / kGtTile;
    w.k_steps = (int)((a.rows + kGtK - 1) / kGtK);
    w.err = a.err;
    const cudaError_t e = launch_gt<T, kGtDx>(x, follows, s);
    return e != cudaSuccess ? e : launch_gt<T, kGtDw>(w, true, s);
}

}  // namespace gs
