// gs_gated_few.cuh -- the gated projections of a few rows, where reading the weights
// is all there is to do.
#pragma once

#include "gs_gated.cuh"

namespace gs {

// 16-bit types.  A block makes eight outputs of up to 8 NB rows: its eight warps share
// the contraction, 32 steps in turn, and join their sums in order.  The matrix
// instruction's sixteen rows are eight of Wg and the same eight of Wu, so a thread ends
// up with G and U of the same outputs.  A sum may take its steps in any order, so a
// lane's 16-byte run of a row serves as it was loaded, in both operands alike.  (The
// tensor cores of a pair of CTAs would read 128 weights at a time and leave most SMs
// without any.)
constexpr int kFewThreads = 256, kFewWarps = kFewThreads / 32, kFewOutputs = 8;
constexpr int kFewMost = 32;   // rows of a block
// Widest rows in 16-bit types: the matrix instruction cuts its sums off as the larger
// tensor cores do, and a warp's run of them is not broken up.
constexpr int kFewWidth = 262144;
// From so many outputs on the large tiles of 64 give every pair of CTAs one; from half as
// many, blocks of eight warps with two each give every SM one.
constexpr int kFewFilled = 4864;
// More than sixteen rows of as many outputs are left to the large tiles: 24 rows, 2048 x
// 8192, bf16 18 us and here 25, fp32 121 and 128 (and 1024 x 4096, bf16 10.5 and 9.7, fp32
// 49 and 44).
template <typename T> bool gated_few_takes(const GatedArgs &a) {
    return a.rows <= (a.F < kFewFilled ? kFewMost : kFewMost / 2) && (sizeof(T) == 4 || a.D <= kFewWidth);
}

template <typename T>
__device__ __forceinline__ void few_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (__is_same(T, __half))
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight elements from d on of a row of D; zeros behind its end and for a row that is
// not there.  RUNS: rows are multiples of 16 bytes and start on one; others are loaded an
// element at a time (8192 outputs bf16, one row of 2048 16 us, of 2047 27; 16 rows 17 and 36).
template <typename T, bool RUNS>
__device__ __forceinline__ uint4 few_load(const T *row, bool here, int d, int D) {
    if (RUNS) return here && d < D ? __ldg(reinterpret_cast<const uint4 *>(row + d)) : uint4();
    uint4 v;
    T *e = reinterpret_cast<T *>(&v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = here && d + i < D ? row[d + i] : IO<T>::st(0.0f);
    return v;
}

// H, and G and U where they are kept, of output f and row r.
template <typename T>
__device__ __forceinline__ void few_store(const GatedArgs &a, const GatedPtrs &p, int64_t r, int f,
                                          float g, float u) {
    const int64_t at = r * a.F + f;
    if (p.bg) {
        g += IO<T>::ld((const T *)p.bg + f);
        u += IO<T>::ld((const T *)p.bu + f);
    }
    if (p.G) {
        ((T *)p.G)[at] = IO<T>::st(g);
        ((T *)p.U)[at] = IO<T>::st(u);
    }
    with_act(a.act, [&](auto act) { g = act_of<T, decltype(act)::value>(g) * u; });
    ((T *)p.H)[at] = IO<T>::st(g);
}

template <typename T, int NB, bool RUNS>
__global__ void __launch_bounds__(kFewThreads) gated_few_kernel(GatedArgs a, GatedPtrs p) {
    __shared__ float4 part[kFewWarps][NB][32];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int f = blockIdx.x * kFewOutputs + lane / 4, at = lane % 4 * 8;
    const T *wg = (const T *)p.Wg + (int64_t)f * a.D, *wu = (const T *)p.Wu + (int64_t)f * a.D;
    float c[NB][4] = {};
#pragma unroll 4
    for (int d = warp * 32 + at; d < a.D + at; d += kFewWarps * 32) {   // whole warps
        const uint4 g = few_load<T, RUNS>(wg, f < a.F, d, a.D), u = few_load<T, RUNS>(wu, f < a.F, d, a.D);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int r = b * 8 + lane / 4;
            const uint4 x = few_load<T, RUNS>((const T *)p.X + (int64_t)r * a.D, r < a.rows, d, a.D);
            few_mma<T>(c[b], g.x, u.x, g.y, u.y, x.x, x.y);
            few_mma<T>(c[b], g.z, u.z, g.w, u.w, x.z, x.w);
        }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) part[warp][b][lane] = make_float4(c[b][0], c[b][1], c[b][2], c[b][3]);
    __syncthreads();
    if (warp >= NB || f >= a.F) return;
    float4 s = part[0][warp][lane];
#pragma unroll
    for (int w = 1; w < kFewWarps; ++w) {
        const float4 t = part[w][warp][lane];
        s.x += t.x;
        s.y += t.y;
        s.z += t.z;
        s.w += t.w;
    }
    const int r = warp * 8 + lane % 4 * 2;
    if (r < a.rows) few_store<T>(a, p, r, f, s.x, s.z);
    if (r + 1 < a.rows) few_store<T>(a, p, r + 1, f, s.y, s.w);
}

// fp32: a warp per O (1 or 2) outputs and up to R rows, V contiguous weights per lane and step.  A
// row's loads serve O outputs: of eight rows they are most of the loads (2048 x 8192, 8 rows,
// 46 us, and 64 with one output a warp; 1024 x 4096 14 and 23; four rows 45 and 38).  More than
// eight rows are R at a time on the grid's y axis, and each reads the weights: 16 rows 84 us.
template <int R, int V, int O>
__global__ void __launch_bounds__(kFewThreads) gated_few_f32_kernel(GatedArgs a, GatedPtrs p) {
    using IOV = Run<float, V>;
    const int lane = threadIdx.x % 32;
    const int f = (blockIdx.x * kFewWarps + threadIdx.x / 32) * O;
    const int64_t r0 = (int64_t)blockIdx.y * R;
    if (f >= a.F) return;
    const float *wg = (const float *)p.Wg + (int64_t)f * a.D, *wu = (const float *)p.Wu + (int64_t)f * a.D;
    const int64_t next = O > 1 && f + 1 < a.F ? a.D : 0;   // to the second output; behind the last, that one
    const float *x = (const float *)p.X + r0 * a.D;
    float g[O][R] = {}, u[O][R] = {};
#pragma unroll O == 1 ? 4 : 2
    for (int d = lane * V; d < a.D; d += 32 * V) {
        float vg[O][V], vu[O][V];
#pragma unroll
        for (int o = 0; o < O; ++o) {
            IOV::widen(IOV::load(wg + o * next + d), vg[o]);
            IOV::widen(IOV::load(wu + o * next + d), vu[o]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float vx[V];
            IOV::widen(r0 + r < a.rows ? IOV::load(x + (int64_t)r * a.D + d) : IOV::zero(), vx);
#pragma unroll
            for (int o = 0; o < O; ++o)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    g[o][r] = fmaf(vg[o][e], vx[e], g[o][r]);
                    u[o][r] = fmaf(vu[o][e], vx[e], u[o][r]);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < O; ++k)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                g[k][r] += __shfl_xor_sync(0xffffffffu, g[k][r], o);
                u[k][r] += __shfl_xor_sync(0xffffffffu, u[k][r], o);
            }
#pragma unroll
    for (int o = 0; o < O; ++o)
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane == o * R + r && r0 + r < a.rows && f + o < a.F)
                few_store<float>(a, p, r0 + r, f + o, g[o][r], u[o][r]);
}

template <typename T> cudaError_t launch_gated_few(const GatedArgs &a, const GatedPtrs &p, cudaStream_t s) {
    const bool runs = a.D % kVec<T> == 0 && aligned16(p.X) && aligned16(p.Wg) && aligned16(p.Wu);
    if constexpr (sizeof(T) == 4) {
        const auto run = [&](auto n, auto outputs) {
            constexpr int R = decltype(n)::value, O = decltype(outputs)::value;
            const auto kernel = runs ? gated_few_f32_kernel<R, 4, O> : gated_few_f32_kernel<R, 1, O>;
            kernel<<<dim3((a.F + kFewWarps * O - 1) / (kFewWarps * O), (unsigned)((a.rows + R - 1) / R)),
                     kFewThreads, 0, s>>>(a, p);
        };
        using std::integral_constant;
        if (a.rows == 1)
            run(integral_constant<int, 1>(), integral_constant<int, 1>());
        else if (a.rows <= 4)
            run(integral_constant<int, 4>(), integral_constant<int, 1>());
        else if (a.F < kFewFilled / 2)
            run(integral_constant<int, 8>(), integral_constant<int, 1>());
        else
            run(integral_constant<int, 8>(), integral_constant<int, 2>());
    } else {
        const unsigned blocks = (a.F + kFewOutputs - 1) / kFewOutputs;
        const auto run = [&](auto n) {
            constexpr int NB = decltype(n)::value;
            const auto kernel = runs ? gated_few_kernel<T, NB, true> : gated_few_kernel<T, NB, false>;
            kernel<<<blocks, kFewThreads, 0, s>>>(a, p);
        };
        if (a.rows <= 8)
            run(std::integral_constant<int, 1>());
        else if (a.rows <= 16)
            run(std::integral_constant<int, 2>());
        else
            run(std::integral_constant<int, 4>());
    }
    return cudaGetLastError();
}

}  // namespace gs
