// gs_residual_norm.cuh -- the norm after a branch, its gate, the scaled residual sum
// and the norm before the next branch, forward and backward.
//
// Forward, per row (fp32 throughout, one rounding at each store):
//   z' = norm(z) * zs + zb, or z;   s = alpha x + gate z';   y = norm(s) * scale + B,
//   norm(v) = (v - mean) / sqrt(var + eps), or v / sqrt(mean v^2 + eps).
// Backward, with N(w, v^, inv) = inv (w - mean w - v^ mean(w v^)):
//   ds = dS + N(dy scale, s^, inv_s), dx = alpha ds, e = gate ds, dz = N(e zs, z^, inv_z),
//   dscale = sum dy s^, dB = sum dy, dzs = sum e z^, dzb = sum e, and per gate
//   dgate = sum ds z' over the rows that share it.
//
// Both read their inputs once: a row stays in the registers of the L threads that
// share it, NV runs of V elements each, up to D = 8192 (backward up to 4096, and to 8192
// with two sums); longer rows are read again for each pass.  Backward, each team of L threads walks segments: rows that share a
// gate, or every chunks-th of them.  A thread keeps the sums of its columns over all
// its rows, and those for the gate over a segment; a second kernel adds the teams'
// sums in order.
#pragma once

#include <algorithm>
#include <initializer_list>

#include "gs_sums.cuh"

namespace gs {

constexpr int kResThreads = 256;       // of a block, at least
constexpr int kResOnChip = 8192;       // widest row held in registers, forward
constexpr int kResStaged = 4096;       // widest row that is staged, backward
constexpr int kResSms = 152;

constexpr int res_block(int L) { return L > kResThreads ? L : kResThreads; }

// Sums of two values over the L threads of a row (a warp or less, or whole warps);
// slots alternate between calls, so that one barrier per call suffices.
template <int L> __device__ __forceinline__ void team_sum2(float &a, float &b, int &slot) {
    if (L < 32) {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        return;
    }
    // the lower half of a warp goes on with a, the upper half with b
    const int lane = threadIdx.x % 32;
    float v = lane < 16 ? a : b;
    v += __shfl_xor_sync(0xffffffffu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (L == 32) {
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
    } else {
        constexpr int W = L > 32 ? L / 32 : 1;
        __shared__ float s[2][2][32];
        if (lane % 16 == 0) s[slot][lane / 16][threadIdx.x / 32] = v;
        __syncthreads();
        a = b = 0.0f;
        const int first = threadIdx.x / L * W;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            a += s[slot][0][first + w];
            b += s[slot][1][first + w];
        }
        slot ^= 1;
    }
}
template <int L> __device__ __forceinline__ float team_sum(float a, int &slot) {
    float none = 0.0f;
    team_sum2<L>(a, none, slot);
    return a;
}

// A row per team of L threads.  Bound by memory where rows are runs (1,048,576 x 64 fp32,
// 1.07 GB, 155 us: 1.03 of a copy's rate; 2048 x 8192 bf16 34 us, 3.9 TB/s), by the
// instructions of pairs and single elements elsewhere (21760 x 771 bf16 62 us, 2.1 TB/s; fp32
// 60, 4.4).
template <typename T, int V, int L, int NV, bool POST>
__global__ void __launch_bounds__(res_block(L)) resnorm_kernel(ResNormArgs a, ResNormPtrs p) {
    using IOV = Run<T, V>;
    constexpr int kTeams = res_block(L) / L;
    const int part = threadIdx.x % L;
    const int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / L;
    const float per_d = 1.0f / (float)a.D;
    typename IOV::Raw rx[NV], rz[NV], rg[NV];
    const int64_t gate =
        a.groups > 1 && row < a.rows ? (int64_t)((uint32_t)row / (uint32_t)a.group_rows) * a.D : 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int d = (k * L + part) * V;
        const bool on = row < a.rows && d < a.D;
        rx[k] = on ? IOV::load((const T *)p.X + row * a.D + d) : IOV::zero();
        rz[k] = on ? IOV::load((const T *)p.Z + row * a.D + d) : IOV::zero();
        if (a.groups > 0) rg[k] = on ? IOV::load((const T *)p.gate + gate + d) : IOV::zero();
    }
    int slot = 0;
    constexpr int N = NV * V, P = (N + 1) / 2;   // a thread's elements, in pairs
    const auto both = [](float x) { return make_float2(x, x); };
    const auto inside = [&](int i) { return (i / V * L + part) * V < a.D; };   // element i
    const auto pairs_of = [](const typename IOV::Raw (&raw)[NV], float2 (&v)[P]) {
        float f[2 * P] = {};
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float x[V];
            IOV::widen(raw[k], x);
#pragma unroll
            for (int e = 0; e < V; ++e) f[k * V + e] = x[e];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    };
    // f(i, w, b) for each pair i of the row's columns with two vectors' elements (zeros of
    // none).  All loads first, but a run at a time in blocks whose threads hold eight:
    // there they do not fit the registers (2048 x 8192 fp32 67 us, and 47 by runs; 32768 x
    // 1024 bf16, a warp per row, 58 us and 96).
    const auto with_params = [&](const void *wp, const void *bp, auto &&f) {
        const auto load = [&](const void *base, int k) {
            const int d = (k * L + part) * V;
            return base && d < a.D ? IOV::load((const T *)base + d) : IOV::zero();
        };
        if constexpr (L == 256 && NV == 8 && V > 2) {
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float w[V], b[V] = {};
                IOV::widen(load(wp, k), w);
                if (bp) IOV::widen(load(bp, k), b);   // a branch, which loads do not move across
#pragma unroll
                for (int h = 0; h < V / 2; ++h)
                    f(k * (V / 2) + h, make_float2(w[2 * h], w[2 * h + 1]),
                      make_float2(b[2 * h], b[2 * h + 1]));
            }
        } else {
            typename IOV::Raw rw[NV], rb[NV];
            float2 w[P], b[P];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                rw[k] = load(wp, k);
                rb[k] = load(bp, k);
            }
            pairs_of(rw, w);
            pairs_of(rb, b);
#pragma unroll
            for (int i = 0; i < P; ++i) f(i, w[i], b[i]);
        }
    };
    const auto put = [&](void *base, const float2 (&v)[P]) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            float x[V];
#pragma unroll
            for (int e = 0; e < V; ++e) x[e] = (k * V + e) % 2 ? v[(k * V + e) / 2].y : v[(k * V + e) / 2].x;
            if (row < a.rows && d < a.D) IOV::store((T *)base + row * a.D + d, x);
        }
    };
    // v minus its mean, and the mean and reciprocal deviation; zeros behind a row's end
    // stay zeros
    const auto normalise = [&](float2 (&v)[P], float &mean, float &inv) {
        mean = 0.0f;
        if (a.layer) {
            float2 t = both(0.0f);
#pragma unroll
            for (int i = 0; i < P; ++i) t = add_f32x2(t, v[i]);
            mean = team_sum<L>(t.x + t.y, slot) * per_d;
#pragma unroll
            for (int i = 0; i < P; ++i)
                v[i] = add_f32x2(v[i], make_float2(inside(2 * i) ? -mean : 0.0f,
                                                   2 * i + 1 < N && inside(2 * i + 1) ? -mean : 0.0f));
        }
        float2 t = both(0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) t = fma_f32x2(v[i], v[i], t);
        inv = 1.0f / sqrtf(fmaf(team_sum<L>(t.x + t.y, slot), per_d, a.eps));
    };
    float2 v[P], x[P];
    float4 stats = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    pairs_of(rz, v);
    if (POST) {
        normalise(v, stats.x, stats.y);
        with_params(p.z_scale, p.z_B, [&](int i, float2 w, float2 b) {
            v[i] = fma_f32x2(mul_f32x2(v[i], both(stats.y)), w, b);
        });
    }
    pairs_of(rx, x);
    if (a.groups > 0) {
        float2 g[P];
        pairs_of(rg, g);
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = fma_f32x2(g[i], v[i], mul_f32x2(x[i], both(a.alpha)));
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = fma_f32x2(x[i], both(a.alpha), v[i]);
    }
    put(p.S, v);
    normalise(v, stats.z, stats.w);
    with_params(p.scale, p.B, [&](int i, float2 w, float2 b) {
        v[i] = fma_f32x2(mul_f32x2(v[i], both(stats.w)), w, b);
    });
    put(p.Y, v);
    if (row < a.rows && part == 0 && p.stats) *reinterpret_cast<float4 *>(p.stats + 4 * row) = stats;
}

// Rows wider than kResOnChip: a block per row that reads it again for each sum.
template <typename T, int V, int L>
__global__ void __launch_bounds__(L) resnorm_wide_kernel(ResNormArgs a, ResNormPtrs p) {
    using IOV = Run<T, V>;
    const int64_t row = blockIdx.x, at = row * a.D;
    const int64_t gate = a.groups > 1 ? row / a.group_rows * a.D : 0;
    const float per_d = 1.0f / (float)a.D;
    int slot = 0;
    const auto get = [](const void *base, int64_t i, float (&v)[V]) {
        IOV::widen(base ? IOV::load((const T *)base + i) : IOV::zero(), v);
    };
    const auto statistics = [&](auto value, float &mean, float &inv) {
        float s = 0.0f, v[V];
        mean = 0.0f;
        if (a.layer) {
#pragma unroll 4
            for (int d = threadIdx.x * V; d < a.D; d += L * V) {
                value(d, v);
#pragma unroll
                for (int e = 0; e < V; ++e) s += v[e];
            }
            mean = team_sum<L>(s, slot) * per_d;
        }
        s = 0.0f;
#pragma unroll 4
        for (int d = threadIdx.x * V; d < a.D; d += L * V) {
            value(d, v);
#pragma unroll
            for (int e = 0; e < V; ++e) s = fmaf(v[e] - mean, v[e] - mean, s);
        }
        inv = 1.0f / sqrtf(fmaf(team_sum<L>(s, slot), per_d, a.eps));
    };
    float4 st = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    if (p.z_scale) statistics([&](int d, float (&v)[V]) { get(p.Z, at + d, v); }, st.x, st.y);
    const auto sum = [&](int d, float (&v)[V]) {
        float x[V];
        get(p.Z, at + d, v);
        if (p.z_scale) {
            float w[V], b[V];
            get(p.z_scale, d, w);
            get(p.z_B, d, b);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf((v[e] - st.x) * st.y, w[e], b[e]);
        }
        get(p.X, at + d, x);
        if (a.groups > 0) {
            float g[V];
            get(p.gate, gate + d, g);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf(g[e], v[e], a.alpha * x[e]);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = fmaf(a.alpha, x[e], v[e]);
        }
    };
    statistics(sum, st.z, st.w);
#pragma unroll 2
    for (int d = threadIdx.x * V; d < a.D; d += L * V) {
        float s[V], w[V], b[V];
        sum(d, s);
        get(p.scale, d, w);
        get(p.B, d, b);
        IOV::store((T *)p.S + at + d, s);
#pragma unroll
        for (int e = 0; e < V; ++e) s[e] = fmaf((s[e] - st.z) * st.w, w[e], b[e]);
        IOV::store((T *)p.Y + at + d, s);
    }
    if (threadIdx.x == 0 && p.stats) *reinterpret_cast<float4 *>(p.stats + 4 * row) = st;
}

// How the backward pass goes over the rows: `teams` walkers in `blocks` blocks;
// group g's rows are cut into `chunks` segments, the c-th of every chunks-th row from
// row c on, and walker w takes segments w, w + teams, ...: `rounds` of them, `steps`
// rows each, at most.  With one chunk the gate's gradient is complete in a walker.
struct ResNormPlan {
    int blocks, teams, groups, chunks, rounds, steps;
    int64_t group_rows;
};
inline ResNormPlan resnorm_plan(const ResNormArgs &a, int teams_per_block, int most_blocks) {
    ResNormPlan q;
    q.groups = a.groups > 0 ? a.groups : 1;
    q.group_rows = a.groups > 0 ? a.group_rows : a.rows;
    const int64_t need = (a.rows + teams_per_block - 1) / teams_per_block;
    q.blocks = (int)(need < most_blocks ? need : most_blocks);
    q.teams = q.blocks * teams_per_block;
    // the fewest rows that a walker takes one after another, with few chunks
    int64_t best = INT64_MAX;
    const int64_t even = q.teams / q.groups, most = even < 8 ? 8 : even;
    q.chunks = 1;
    for (int64_t c = 1; c <= most && c <= q.group_rows; c = c < 8 || c == most ? c + 1 : most) {
        if (c > 1 && q.groups * c > 4 * (int64_t)q.teams) break;   // each chunk leaves D sums behind
        const int64_t rounds = (q.groups * c + q.teams - 1) / q.teams;
        const int64_t cost = rounds * ((q.group_rows + c - 1) / c);
        if (cost < best) {
            best = cost;
            q.chunks = (int)c;
        }
    }
    q.rounds = (int)(((int64_t)q.groups * q.chunks + q.teams - 1) / q.teams);
    q.steps = (int)((q.group_rows + q.chunks - 1) / q.chunks);
    return q;
}

// A walker's place: segment, step in it, the row there (-1: none) and its gate.
struct ResNormWalk {
    uint32_t segment, gate;
    int row, step;
    __device__ __forceinline__ void start(const ResNormPlan &q, uint32_t s, int i = 0) {
        segment = s;
        step = i;
        gate = s / (uint32_t)q.chunks;
        const int64_t within = s - gate * (uint32_t)q.chunks + (int64_t)i * q.chunks;
        row = gate < (uint32_t)q.groups && within < q.group_rows ? (int)(gate * q.group_rows + within) : -1;
    }
    __device__ __forceinline__ void next(const ResNormPlan &q) {
        if (++step < q.steps) {
            if (row >= 0) {
                const int64_t to = (int64_t)row + q.chunks;
                row = to < (gate + (int64_t)1) * q.group_rows ? (int)to : -1;
            }
        } else {
            start(q, segment + q.teams);
        }
    }
};

// Blocks per SM, by the elements of a row that a thread holds.
constexpr int resnorm_backward_blocks(int L, int N) {
    return L > kResThreads ? 1 : N <= 4 ? 3 : N <= 8 ? 2 : 1;
}

// 65536 x 256 bf16, all sums, 201 MB in 48 us, 4.2 TB/s; 266305 x 63 in 109, 1.8 TB/s.
// dX, dZ and, into partials[block][vector], the block's column sums (for dScale, dB
// and, with POST, dz_scale and dz_B); into gate_partials[segment] those for the gate, or
// [block] where all rows share one.  The next row's loads are issued before this one is
// worked on.
template <typename T, int V, int L, int NV, bool POST, bool GATE>
__global__ void __launch_bounds__(res_block(L), resnorm_backward_blocks(L, NV * V))
    resnorm_backward_kernel(ResNormArgs a, ResNormPtrs p, ResNormPlan q, float *partials,
                            float *gate_partials) {
    using IOV = Run<T, V>;
    constexpr int kThreads = res_block(L), kTeams = kThreads / L, kVectors = POST ? 4 : 2;
    const int part = threadIdx.x % L, team = threadIdx.x / L;
    const float per_d = 1.0f / (float)a.D;
    float sum[kVectors][NV][V] = {}, gate_sum[NV][V] = {};
    typename IOV::Raw rd[NV], ry[NV], rs[NV], rz[NV], rg[NV];
    float4 st;
    const auto load = [&](const ResNormWalk &w) {
        const int64_t row = w.row, at = row * a.D, gate = (int64_t)w.gate * a.D;
        const bool here = row >= 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = here && d < a.D;
            rd[k] = on && p.dS ? IOV::load((const T *)p.dS + at + d) : IOV::zero();
            ry[k] = on ? IOV::load((const T *)p.dY + at + d) : IOV::zero();
            rs[k] = on ? IOV::load((const T *)p.S + at + d) : IOV::zero();
            rz[k] = on ? IOV::load((const T *)p.Z + at + d) : IOV::zero();
            if (GATE) rg[k] = on ? IOV::load((const T *)p.gate + gate + d) : IOV::zero();
        }
        st = here ? __ldg(reinterpret_cast<const float4 *>(p.stats) + row)
                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    };
    ResNormWalk w;
    w.start(q, blockIdx.x * kTeams + team);
    load(w);
    int slot = 0;
    for (int64_t n = (int64_t)q.rounds * q.steps; n > 0; --n) {
        const int64_t row = w.row, segment = w.segment;
        const bool ends = w.step + 1 == q.steps;
        float sh[NV][V], wy[NV][V], ds[NV][V], zh[NV][V], gate[NV][V];
        float t0 = 0.0f, t1 = 0.0f;
        const float4 now = st;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = d < a.D;
            float y[V], c[V];
            IOV::widen(rs[k], sh[k]);
            IOV::widen(ry[k], y);
            IOV::widen(on ? IOV::load((const T *)p.scale + d) : IOV::zero(), c);
            IOV::widen(rd[k], ds[k]);
            IOV::widen(rz[k], zh[k]);
            if (GATE) IOV::widen(rg[k], gate[k]);
            // zeros behind a row's end, whose products and sums are zeros
            const float m = on ? now.z : 0.0f, i = on ? now.w : 0.0f;
            const float mz = on ? now.x : 0.0f, iz = on ? now.y : 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sh[k][e] = (sh[k][e] - m) * i;
                sum[0][k][e] = fmaf(y[e], sh[k][e], sum[0][k][e]);
                sum[1][k][e] += y[e];
                wy[k][e] = y[e] * c[e];
                t0 += wy[k][e];
                t1 = fmaf(wy[k][e], sh[k][e], t1);
                if (POST) zh[k][e] = (zh[k][e] - mz) * iz;
            }
        }
        w.next(q);
        load(w);
        team_sum2<L>(t0, t1, slot);
        t0 = a.layer ? t0 * -per_d : 0.0f;
        t1 *= -per_d;
        float u0 = 0.0f, u1 = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = d < a.D;
            float c[V], b[V] = {}, out[V];
            if (POST) {
                IOV::widen(on ? IOV::load((const T *)p.z_scale + d) : IOV::zero(), c);
                if (GATE && p.z_B) IOV::widen(on ? IOV::load((const T *)p.z_B + d) : IOV::zero(), b);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
                ds[k][e] = fmaf(fmaf(sh[k][e], t1, wy[k][e] + t0), now.w, ds[k][e]);
                out[e] = a.alpha * ds[k][e];
                if (GATE) {
                    gate_sum[k][e] =
                        fmaf(ds[k][e], POST ? fmaf(zh[k][e], c[e], b[e]) : zh[k][e], gate_sum[k][e]);
                    ds[k][e] *= gate[k][e];
                }
                if (POST) {
                    sum[kVectors - 2][k][e] = fmaf(ds[k][e], zh[k][e], sum[kVectors - 2][k][e]);
                    sum[kVectors - 1][k][e] += ds[k][e];
                    ds[k][e] *= c[e];
                    u0 += ds[k][e];
                    u1 = fmaf(ds[k][e], zh[k][e], u1);
                }
            }
            if (row >= 0 && on) {
                IOV::store((T *)p.dX + row * a.D + d, out);
                if (!POST) IOV::store((T *)p.dZ + row * a.D + d, ds[k]);
            }
        }
        if (POST) {
            team_sum2<L>(u0, u1, slot);
            u0 = a.layer ? u0 * -per_d : 0.0f;
            u1 *= -per_d;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int d = (k * L + part) * V;
                float out[V];
#pragma unroll
                for (int e = 0; e < V; ++e) out[e] = fmaf(zh[k][e], u1, ds[k][e] + u0) * now.y;
                if (row >= 0 && d < a.D) IOV::store((T *)p.dZ + row * a.D + d, out);
            }
        }
        if (GATE && ends && q.groups > 1) {
            if (segment < (int64_t)q.groups * q.chunks) {
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    const int d = (k * L + part) * V;
                    if (d >= a.D) continue;
                    if (q.chunks == 1) {
                        IOV::store((T *)p.dgate + segment * a.D + d, gate_sum[k]);
                    } else {
#pragma unroll
                        for (int e = 0; e < V; ++e) gate_partials[segment * a.D + d + e] = gate_sum[k][e];
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) gate_sum[k][e] = 0.0f;
        }
    }
    // the teams of the block in order, one vector and run at a time
    __shared__ float join[kTeams > 1 ? kThreads * V : 1];
    const auto leave = [&](const float (&sums)[NV][V], float *out) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (kTeams > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < V; ++e) join[threadIdx.x * V + e] = sums[k][e];
                __syncthreads();
                for (int c = threadIdx.x; c < L * V; c += kThreads) {
                    const int d = k * L * V + c;
                    float t = 0.0f;
#pragma unroll
                    for (int g = 0; g < kTeams; ++g) t += join[g * L * V + c];
                    if (d < a.D) out[d] = t;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int d = (k * L + part) * V + e;
                    if (d < a.D) out[d] = sums[k][e];
                }
            }
        }
    };
    if (GATE && q.groups == 1) leave(gate_sum, gate_partials + (int64_t)blockIdx.x * a.D);
    if (!partials) return;
#pragma unroll
    for (int j = 0; j < kVectors; ++j)
        leave(sum[j], partials + ((int64_t)blockIdx.x * kVectors + j) * a.D);
}

// ------------------------------------------------------------------ backward, staged

// Rows wider than a warp's run: each team's rows come to shared memory by bulk copies
// that its first threads issue, one array each, as many rows ahead as there is room
// for, so that the registers hold sums and not loads in flight.  A block of 512 threads
// per SM.  Bound by the latency of a row's two sums and by instruction issue (44 % of the
// slots): 16384 x 1024 bf16, all sums, sixteen gates, 201 MB in 53 us, 3.8 TB/s; 5003 x 771
// fp32 in 21 us, 4.3 TB/s.
constexpr int kStagedThreads = 512;
constexpr int kStagedRing = 200 * 1024;   // bytes of all teams' rows, and of their totals
constexpr int kStagedN = 8;               // elements of a thread
constexpr int kStagedMost = 4;            // rows of a team, being worked on and ahead

// Bytes of one array's row: it starts on a 16-byte boundary of memory, up to 15 bytes
// ahead of its first element.
constexpr int staged_pitch(int D, int size) { return (D * size + 15 + 15) / 16 * 16; }

// Arrays of a stage, and behind them the row's statistics and its place: row (-1: none),
// gate, segment (-1: none), whether the segment ends with it.
constexpr int kStagedStats = 32;
struct StagedShape {
    int stages, pitch, arrays;
};
// Floats of the totals that a team keeps over its gates (dz_scale's and dz_B's).
constexpr int staged_totals(bool post, bool gate) { return post && gate ? 2 * kStagedN * kStagedThreads : 0; }
constexpr StagedShape staged_shape(int D, int size, int L, bool post, bool gate, bool dS) {
    StagedShape q = {};
    q.pitch = staged_pitch(D, size);
    q.arrays = 3 + dS + gate;
    const int per = kStagedThreads / L * (q.arrays * q.pitch + kStagedStats);
    const int room = (kStagedRing - 4 * staged_totals(post, gate)) / per;
    q.stages = room < kStagedMost ? room : kStagedMost;
    return q;
}

// Barrier of a team of whole warps.
template <int L> __device__ __forceinline__ void team_barrier() {
    if (L == 32)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.x / L + 1), "n"(L) : "memory");
}
template <int L>
__device__ __forceinline__ void staged_sum2(float &a, float &b, float (*shared)[2][L / 32], int &slot) {
    const int lane = threadIdx.x % 32;
    float v = lane < 16 ? a : b;
    v += __shfl_xor_sync(0xffffffffu, lane < 16 ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (L == 32) {
        a = __shfl_sync(0xffffffffu, v, 0);
        b = __shfl_sync(0xffffffffu, v, 16);
        return;
    }
    if (lane % 16 == 0) shared[slot][lane / 16][threadIdx.x % L / 32] = v;
    team_barrier<L>();
    const float2 *sa = reinterpret_cast<const float2 *>(shared[slot][0]);
    const float2 *sb = reinterpret_cast<const float2 *>(shared[slot][1]);
    float2 ta = sa[0], tb = sb[0];
#pragma unroll
    for (int w = 1; w < L / 64; ++w) {
        ta = add_f32x2(ta, sa[w]);
        tb = add_f32x2(tb, sb[w]);
    }
    a = ta.x + ta.y;
    b = tb.x + tb.y;
    slot ^= 1;
}

// A row of D elements at `from` to `to`, from the 16-byte boundary at or before its
// start to the one at or after its end, and this thread's arrival on `bar`.  With EDGES,
// `first` and `last` bound the tensor, whose outermost elements are copied one at a time
// where a boundary lies outside.
template <typename T, bool EDGES>
__device__ __forceinline__ void staged_fetch(unsigned char *to, const T *from, int D, const T *first,
                                             const T *last, uint64_t *bar) {
    const uintptr_t start = (uintptr_t)from & ~(uintptr_t)15;
    uintptr_t a = start, b = ((uintptr_t)(from + D) + 15) & ~(uintptr_t)15;
    if (EDGES && (a < (uintptr_t)first || b > (uintptr_t)last)) {
        if (a < (uintptr_t)first) a += 16;
        if (b > (uintptr_t)last) b -= 16;
        if (b < a) b = a;
        T *row = reinterpret_cast<T *>(to + ((uintptr_t)from & 15));
        for (int d = 0; d < D && (uintptr_t)(from + d) < a; ++d) row[d] = from[d];
        for (int d = D - 1; d >= 0 && (uintptr_t)(from + d) >= b; --d) row[d] = from[d];
        fence_proxy_async_smem();   // before this thread's later copies to the same place
    }
    const uint32_t bytes = (uint32_t)(b - a);
    mbar_arrive_expect_tx(bar, bytes);
    if (bytes) bulk_copy_g2s(to + (a - start), reinterpret_cast<const void *>(a), bytes, bar);
}

// The sums of ds and of ds * z^ over the rows that share a gate give the gradients of all
// that stands between z^ and S: dgate = zs * sum ds z^ + zb * sum ds, and with the gate
// as a factor they add up to dzs and dzb over the gates.
template <typename T, int V, int L, int NV, bool POST, bool GATE>
__global__ void __launch_bounds__(kStagedThreads, 1)
    resnorm_staged_kernel(ResNormArgs a, ResNormPtrs p, ResNormPlan q, StagedShape sh_, float *partials,
                          float *gate_partials) {
    constexpr int kTeams = kStagedThreads / L, N = NV * V, P = N / 2, kVectors = POST ? 4 : 2;
    using IOV = Run<T, V>;
    constexpr bool kWhole = V * sizeof(T) == 16;   // rows start on 16-byte boundaries
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ __align__(8) uint64_t full[kTeams][kStagedMost];
    __shared__ __align__(16) float shared_sums[kTeams][2][2][L / 32];
    const int part = threadIdx.x % L, team = threadIdx.x / L;
    const int stages = sh_.stages, row_bytes = sh_.pitch, stats_at = sh_.arrays * row_bytes;
    const int stage_bytes = stats_at + kStagedStats;   // a multiple of 16
    static_assert(N <= kStagedN && N % 2 == 0, "elements of a thread");
    constexpr int kTotals = POST && GATE ? 2 * N * kStagedThreads : 0;
    // this thread's totals, kStagedThreads floats apart
    float *totals = reinterpret_cast<float *>(ring) + threadIdx.x;
    unsigned char *mine = ring + kTotals * 4 + (size_t)team * stages * stage_bytes;
    float(*sums)[2][L / 32] = shared_sums[team];
    const float per_d = 1.0f / (float)a.D;
    const int zs_at = 2, gate_at = 3, ds_at = GATE ? 4 : 3;   // dY and S are the first two

    if (part == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[team][s], sh_.arrays + 1);
        fence_mbar_init();
    }
    team_barrier<L>();

    // the row that is fetched next; the arrays, and the statistics after them, go round
    // the warps, so that none of them holds up the others
    ResNormWalk ahead;
    ahead.start(q, blockIdx.x * kTeams + team);
    const int steps = q.rounds * q.steps;
    const int mine_of = part % 32 * (L / 32) + part / 32;
    const bool fetches = mine_of < sh_.arrays, of_gate = GATE && mine_of == gate_at;
    const T *array = (const T *)(mine_of == 0       ? p.dY
                                 : mine_of == 1     ? p.S
                                 : mine_of == zs_at ? p.Z
                                 : of_gate          ? p.gate
                                                    : p.dS);
    const T *array_end = array + (of_gate ? q.groups : a.rows) * (int64_t)a.D;
    const auto fetch = [&](int s) {   // into stage s
        uint64_t *bar = &full[team][s];
        if (mine_of == sh_.arrays) {
            unsigned char *to = mine + s * stage_bytes + stats_at;
            *reinterpret_cast<int4 *>(to + 16) = make_int4(
                ahead.row, (int)ahead.gate,
                ahead.segment < (uint32_t)q.groups * q.chunks ? (int)ahead.segment : -1,
                ahead.step + 1 == q.steps);
            mbar_arrive_expect_tx(bar, ahead.row >= 0 ? 16 : 0);
            if (ahead.row >= 0) bulk_copy_g2s(to, p.stats + (int64_t)ahead.row * 4, 16, bar);
        } else if (fetches && ahead.row >= 0)
            staged_fetch<T, !kWhole>(mine + s * stage_bytes + mine_of * row_bytes,
                                    array + (of_gate ? (int64_t)ahead.gate : (int64_t)ahead.row) * a.D, a.D,
                                    array, array_end, bar);
        else if (fetches)   // no row: the phase is over at once
            mbar_arrive(bar);
        ahead.next(q);
    };
    for (int n = 0; n < stages && n < steps; ++n) fetch(n);

    // over all rows, for dScale and dB; over a segment's, of ds * z^ and of ds
    float2 sum[2][P] = {}, seg[2][P] = {};
    if (kTotals)
#pragma unroll
        for (int i = 0; i < 2 * N; ++i) totals[i * kStagedThreads] = 0.0f;
    // a thread's elements of a staged row, in pairs; zeros behind the row's end
    const auto take = [&](const unsigned char *row, const void *base, int64_t offset, float2 (&v)[P]) {
        const T *e = reinterpret_cast<const T *>(
            kWhole ? row : row + ((uintptr_t)((const T *)base + offset) & 15));
        float f[N];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            float x[V];
            IOV::widen(d < a.D ? IOV::load(e + d) : IOV::zero(), x);
#pragma unroll
            for (int i = 0; i < V; ++i) f[k * V + i] = x[i];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    };
    const auto param = [&](const void *base, float2 (&v)[P], int64_t at = 0) {   // of the row's columns
        float f[N];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            float x[V];
            IOV::widen(d < a.D ? IOV::load((const T *)base + at + d) : IOV::zero(), x);
#pragma unroll
            for (int i = 0; i < V; ++i) f[k * V + i] = x[i];
        }
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    };
    const auto element = [](const float2 (&v)[P], int i) { return i % 2 ? v[i / 2].y : v[i / 2].x; };
    const auto put = [&](void *base, int64_t at, const float2 (&v)[P]) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            float x[V];
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = element(v, k * V + i);
            if (d < a.D) IOV::store((T *)base + at + d, x);
        }
    };
    const auto both = [](float x) { return make_float2(x, x); };
    // (v - mean) * inv; behind the row's end 0, whatever the statistics
    const auto normal = [&](float2 (&v)[P], float mean, float inv) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if constexpr (V > 1) {   // a run is inside or outside as a whole
                const bool in = (2 * i / V * L + part) * V < a.D;
                v[i] = mul_f32x2(add_f32x2(v[i], both(in ? -mean : 0.0f)), both(in ? inv : 0.0f));
            } else {
                v[i] = mul_f32x2(add_f32x2(v[i], both(-mean)), both(inv));
                if (2 * i * L + part >= a.D) v[i].x = 0.0f;
                if ((2 * i + 1) * L + part >= a.D) v[i].y = 0.0f;
            }
        }
    };

    // The gate's gradient from a segment's sums, whose share of dz_scale and dz_B is added to
    // the totals.
    const auto gate_sums = [&](float2 (&d)[P], int gate) {
#pragma unroll
        for (int i = 0; i < P; ++i) d[i] = seg[0][i];
        if (POST) {
            float2 g[P], c[P], b[P];
            param(p.gate, g, (int64_t)gate * a.D);
            param(p.z_scale, c);
            if (p.z_B) param(p.z_B, b);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                d[i] = mul_f32x2(seg[0][i], c[i]);
                if (p.z_B) d[i] = fma_f32x2(seg[1][i], b[i], d[i]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float *t = totals + (j * N + 2 * i) * kStagedThreads;
                    t[0] = fmaf(seg[j][i].x, g[i].x, t[0]);
                    t[kStagedThreads] = fmaf(seg[j][i].y, g[i].y, t[kStagedThreads]);
                }
            }
        }
    };

    bool ok = true;
    int slot = 0, s = 0;
    uint32_t parity = 0;
    for (int n = 0; n < steps; ++n) {
        const unsigned char *here = mine + s * stage_bytes;
        float2 sh[P], wy[P], ds[P], zh[P], g[P], c[P];
        param(p.scale, c);
        if (ok) ok = mbar_wait_bounded(&full[team][s], parity, a.err);
        int4 place = *reinterpret_cast<const int4 *>(here + stats_at + 16);
        if (!ok) place = make_int4(-1, 0, -1, 0);
        const int row = place.x;
        const int64_t at = (int64_t)row * a.D;
        float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float2 t0 = both(0.0f), t1 = both(0.0f);
        if (row >= 0) {
            st = *reinterpret_cast<const float4 *>(here + stats_at);
            take(here + row_bytes, p.S, at, sh);
            take(here, p.dY, at, wy);
            normal(sh, st.z, st.w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                sum[0][i] = fma_f32x2(wy[i], sh[i], sum[0][i]);
                sum[1][i] = add_f32x2(sum[1][i], wy[i]);
                wy[i] = mul_f32x2(wy[i], c[i]);
                t0 = add_f32x2(t0, wy[i]);
                t1 = fma_f32x2(wy[i], sh[i], t1);
            }
        }
        float s0 = t0.x + t0.y, s1 = t1.x + t1.y;
        if (POST) param(p.z_scale, c);
        staged_sum2<L>(s0, s1, sums, slot);
        if (L == 32) __syncwarp();
        // the team is past its reads of the row before: that stage is filled again
        if (n > 0 && n - 1 + stages < steps) fetch(s == 0 ? stages - 1 : s - 1);
        s0 = a.layer ? s0 * -per_d : 0.0f;
        s1 *= -per_d;
        float2 u0 = both(0.0f), u1 = both(0.0f);
        if (row >= 0) {
            if (p.dS) {
                take(here + ds_at * row_bytes, p.dS, at, ds);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) ds[i] = both(0.0f);
            }
            take(here + zs_at * row_bytes, p.Z, at, zh);
            if (POST) normal(zh, st.x, st.y);
            float2 out[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                ds[i] = fma_f32x2(fma_f32x2(sh[i], both(s1), add_f32x2(wy[i], both(s0))), both(st.w), ds[i]);
                out[i] = mul_f32x2(ds[i], both(a.alpha));
            }
            put(p.dX, at, out);
            if (GATE) take(here + gate_at * row_bytes, p.gate, (int64_t)place.y * a.D, g);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (POST || GATE) seg[0][i] = fma_f32x2(ds[i], zh[i], seg[0][i]);
                if (POST) seg[1][i] = add_f32x2(seg[1][i], ds[i]);
                if (GATE) ds[i] = mul_f32x2(ds[i], g[i]);
                if (POST) {
                    ds[i] = mul_f32x2(ds[i], c[i]);
                    u0 = add_f32x2(u0, ds[i]);
                    u1 = fma_f32x2(ds[i], zh[i], u1);
                }
            }
            if (!POST) put(p.dZ, at, ds);
        }
        if (POST) {
            s0 = u0.x + u0.y;
            s1 = u1.x + u1.y;
            staged_sum2<L>(s0, s1, sums, slot);
            s0 = a.layer ? s0 * -per_d : 0.0f;
            s1 *= -per_d;
            if (row >= 0) {
                float2 out[P];
#pragma unroll
                for (int i = 0; i < P; ++i)
                    out[i] = mul_f32x2(fma_f32x2(zh[i], both(s1), add_f32x2(ds[i], both(s0))), both(st.y));
                put(p.dZ, at, out);
            }
        }
        if (GATE && place.w && q.groups > 1) {
            if (place.z >= 0) {
                float2 d[P];
                gate_sums(d, place.y);
                if (q.chunks == 1) {
                    put(p.dgate, (int64_t)place.z * a.D, d);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int e = (i / V * L + part) * V + i % V;
                        if (e < a.D) gate_partials[(int64_t)place.z * a.D + e] = element(d, i);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) seg[0][i] = seg[1][i] = both(0.0f);
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    // copies that a wait gave up on land before the block may leave
    if (!ok && part == 0)
        for (int n = steps > stages ? steps - stages : 0; n < steps; ++n)
            mbar_wait_bounded(&full[team][n % stages], (n / stages) & 1, a.err);
    // the teams of the block in order, one vector at a time, by way of the ring
    float *join = reinterpret_cast<float *>(ring) + kTotals;
    const auto leave = [&](const float (&x)[N], float *out) {
        if (kTeams == 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int d = (i / V * L + part) * V + i % V;
                if (d < a.D) out[d] = x[i];
            }
            return;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) join[(team * N + i) * L + part] = x[i];
        __syncthreads();
        for (int c = threadIdx.x; c < N * L; c += kStagedThreads) {
            const int i = c / L, d = (i / V * L + c % L) * V + i % V;
            float t = 0.0f;
#pragma unroll
            for (int g = 0; g < kTeams; ++g) t += join[g * N * L + c];
            if (d < a.D) out[d] = t;
        }
    };
    float x[N];
    if (GATE && q.groups == 1) {   // one segment of all the team's rows
        float2 d[P];
        gate_sums(d, 0);
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = element(d, i);
        leave(x, gate_partials + (int64_t)blockIdx.x * a.D);
    }
    if (!partials) return;
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            x[i] = j < 2 ? element(sum[j % 2], i)
                   : kTotals ? totals[((j % 2) * N + i) * kStagedThreads]
                             : element(seg[j % 2], i);
        leave(x, partials + ((int64_t)blockIdx.x * kVectors + j) * a.D);
    }
}

// Wide rows (resnorm_wide): a block per row for dX and dZ, which leaves the row's two
// means in `means`; then a thread per run of columns for the sums, which reads the inputs
// once more: 10 rows of traffic instead of 6, at 3.8 TB/s in bf16 and 5.0 in fp32 (2048 x
// 8192 with all sums, 48 + 34 us and 79 + 48).
template <typename T, int V, int L>
__global__ void __launch_bounds__(L)
    resnorm_wide_backward_kernel(ResNormArgs a, ResNormPtrs p, float2 *means) {
    using IOV = Run<T, V>;
    const int64_t row = blockIdx.x, at = row * a.D;
    const int64_t gate = a.groups > 1 ? row / a.group_rows * a.D : 0;
    const float4 st = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
    const float per_d = 1.0f / (float)a.D;
    int slot = 0;
    const auto get = [](const void *base, int64_t i, float (&v)[V]) {
        IOV::widen(base ? IOV::load((const T *)base + i) : IOV::zero(), v);
    };
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll 4
    for (int d = threadIdx.x * V; d < a.D; d += L * V) {
        float y[V], c[V], s[V];
        get(p.dY, at + d, y);
        get(p.S, at + d, s);
        get(p.scale, d, c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float w = y[e] * c[e];
            t0 += w;
            t1 = fmaf(w, (s[e] - st.z) * st.w, t1);
        }
    }
    team_sum2<L>(t0, t1, slot);
    t0 = a.layer ? t0 * -per_d : 0.0f;
    t1 *= -per_d;
    if (threadIdx.x == 0) means[row] = make_float2(t0, t1);
    const auto ds_of = [&](int d, float (&ds)[V]) {
        float y[V], c[V], s[V];
        get(p.dY, at + d, y);
        get(p.S, at + d, s);
        get(p.dS, at + d, ds);
        get(p.scale, d, c);
#pragma unroll
        for (int e = 0; e < V; ++e)
            ds[e] = fmaf(fmaf((s[e] - st.z) * st.w, t1, fmaf(y[e], c[e], t0)), st.w, ds[e]);
    };
    const auto to_z = [&](int d, float (&v)[V]) {   // from ds
        float g[V];
        if (a.groups > 0) {
            get(p.gate, gate + d, g);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= g[e];
        }
        if (p.z_scale) {
            get(p.z_scale, d, g);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= g[e];
        }
    };
    float u0 = 0.0f, u1 = 0.0f;
#pragma unroll 2
    for (int d = threadIdx.x * V; d < a.D; d += L * V) {
        float v[V], out[V], z[V];
        ds_of(d, v);
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = a.alpha * v[e];
        IOV::store((T *)p.dX + at + d, out);
        to_z(d, v);
        if (p.z_scale) {
            get(p.Z, at + d, z);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                u0 += v[e];
                u1 = fmaf(v[e], (z[e] - st.x) * st.y, u1);
            }
        } else {
            IOV::store((T *)p.dZ + at + d, v);
        }
    }
    if (!p.z_scale) return;
    team_sum2<L>(u0, u1, slot);
    u0 = a.layer ? u0 * -per_d : 0.0f;
    u1 *= -per_d;
#pragma unroll 2
    for (int d = threadIdx.x * V; d < a.D; d += L * V) {
        float v[V], z[V];
        ds_of(d, v);
        to_z(d, v);
        get(p.Z, at + d, z);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf((z[e] - st.x) * st.y, u1, v[e] + u0) * st.y;
        IOV::store((T *)p.dZ + at + d, v);
    }
}

// Blocks of the sums per SM, and over the columns.
template <int V> constexpr int kResSumsBlocks = V <= 2 ? 6 / V : 2;
inline int resnorm_sums_columns(int D, int V) { return (D + kResThreads * V - 1) / (kResThreads * V); }
template <typename T, int V>
__global__ void __launch_bounds__(kResThreads, kResSumsBlocks<V>)
    resnorm_wide_sums_kernel(ResNormArgs a, ResNormPtrs p, ResNormPlan q, const float2 *means,
                             float *partials, float *gate_partials) {
    using IOV = Run<T, V>;
    wait_for_previous_kernel(means);
    const int d = (blockIdx.x * kResThreads + threadIdx.x) * V;
    if (d >= a.D) return;
    const auto get = [](const void *base, int64_t i, float (&v)[V]) {
        IOV::widen(base ? IOV::load((const T *)base + i) : IOV::zero(), v);
    };
    float scale[V], zs[V], zb[V], sum[4][V] = {}, gate_sum[V] = {};
    get(p.scale, d, scale);
    get(p.z_scale, d, zs);
    get(p.z_B, d, zb);
    if (!p.z_scale)
#pragma unroll
        for (int e = 0; e < V; ++e) zs[e] = 1.0f;
    for (int64_t segment = blockIdx.y; segment < (int64_t)q.groups * q.chunks; segment += q.teams) {
        const int64_t gate = segment / q.chunks, c = segment - gate * q.chunks;
        const int64_t row0 = gate * q.group_rows + c;
        int64_t at = row0 * a.D + d;
        const float4 *stats = reinterpret_cast<const float4 *>(p.stats) + row0;
        const float2 *mean = means + row0;
        float g[V];
        get(a.groups > 0 ? p.gate : nullptr, gate * a.D + d, g);
        const int rows = (int)((q.group_rows - c + q.chunks - 1) / q.chunks);
        const int64_t step = (int64_t)q.chunks * a.D;
#pragma unroll V == 1 ? 4 : 2
        for (int i = 0; i < rows; ++i, at += step, stats += q.chunks, mean += q.chunks) {
            float y[V], s[V], z[V], ds[V];
            get(p.dY, at, y);
            get(p.S, at, s);
            get(p.Z, at, z);
            get(p.dS, at, ds);
            const float4 st = __ldg(stats);
            const float2 t = __ldg(mean);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float sh = (s[e] - st.z) * st.w, zh = (z[e] - st.x) * st.y;
                float v = fmaf(fmaf(sh, t.y, fmaf(y[e], scale[e], t.x)), st.w, ds[e]);
                sum[0][e] = fmaf(y[e], sh, sum[0][e]);
                sum[1][e] += y[e];
                if (a.groups > 0) {
                    gate_sum[e] = fmaf(v, fmaf(zh, zs[e], zb[e]), gate_sum[e]);
                    v *= g[e];
                }
                sum[2][e] = fmaf(v, zh, sum[2][e]);
                sum[3][e] += v;
            }
        }
        if (a.groups > 0) {
            if (q.chunks == 1) {
                IOV::store((T *)p.dgate + segment * a.D + d, gate_sum);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) gate_partials[segment * a.D + d + e] = gate_sum[e];
            }
#pragma unroll
            for (int e = 0; e < V; ++e) gate_sum[e] = 0.0f;
        }
    }
    if (!partials) return;
    const int vectors = p.z_scale ? 4 : 2;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (j < vectors) partials[((int64_t)blockIdx.y * vectors + j) * a.D + d + e] = sum[j][e];
}

// Rows that are read more than once by 512 threads and not 256: of more than 32 KB, so that
// fewer of them are on their way through L2 at once (backward, 838 x 20001 bf16 159 us, and
// 239 by 256; 2048 x 8192 61 and 47).
template <typename T> bool resnorm_large(const ResNormArgs &a) { return a.D * sizeof(T) > 32768; }

// Calls f(L, NV) with the threads per row and the runs per thread of the forward
// pass for a row of `runs` runs.
// Enough elements per thread that its sums' shuffles and barriers do not lead, few of them
// behind the row's end (130055 x 129 bf16 66 us; 331 by 256 threads of one element each, 87
// by a warp of eight; 32263 x 520 fp32 51, and 96 by 256 threads of one run).
template <int V, typename F> cudaError_t resnorm_shape(int runs, F &&f) {
    using std::integral_constant;
    if constexpr (V <= 2) {
#define GS_SHAPE(L, N) \
    if (runs * V <= L * N) return f(integral_constant<int, L>(), integral_constant<int, N / V>());
        GS_SHAPE(8, 4) GS_SHAPE(8, 6) GS_SHAPE(8, 8) GS_SHAPE(16, 6) GS_SHAPE(16, 8) GS_SHAPE(32, 6)
        GS_SHAPE(32, 8) GS_SHAPE(32, 12) GS_SHAPE(32, 16) GS_SHAPE(64, 12) GS_SHAPE(64, 16)
        GS_SHAPE(128, 12) GS_SHAPE(128, 16) GS_SHAPE(256, 12) GS_SHAPE(256, 16) GS_SHAPE(256, 24)
        GS_SHAPE(256, 32)
#undef GS_SHAPE
    } else {
#define GS_SHAPE(L, NV) \
    if (runs <= L * NV) return f(integral_constant<int, L>(), integral_constant<int, NV>());
        GS_SHAPE(4, 1) GS_SHAPE(8, 1) GS_SHAPE(16, 1) GS_SHAPE(32, 1) GS_SHAPE(32, 2) GS_SHAPE(32, 3)
        GS_SHAPE(32, 4) GS_SHAPE(64, 3) GS_SHAPE(64, 4) GS_SHAPE(128, 3) GS_SHAPE(128, 4)
        GS_SHAPE(256, 3) GS_SHAPE(256, 4)
        if constexpr (V == 4) {
            GS_SHAPE(256, 6) GS_SHAPE(256, 8)
        }
#undef GS_SHAPE
    }
    return cudaErrorInvalidValue;   // not reached: D <= kResOnChip
}

// The same for the backward pass: f(staged, L, NV).  A team's sums, five per element, stay
// in registers, up to eight elements of a thread where rows are staged.  Rows of a warp's run
// or less keep their loads in registers: a bulk copy of 128 bytes costs as much to issue as
// one of a few KB (508400 x 33 bf16 117 us, staged 481; 83886 x 200 130 and 64).  MORE: there
// are more than two sums, and rows wider than kResStaged are read again (resnorm_wide).
template <int V, bool MORE, typename F> cudaError_t resnorm_backward_shape(int D, F &&f) {
    using std::integral_constant;
    using std::false_type;
    using std::true_type;
    constexpr int NV = kStagedN / V;
    if constexpr (V <= 2) {
#define GS_SHAPE(STAGED, L, N)        \
    if constexpr (N % V == 0)         \
        if (D <= L * N) return f(STAGED(), integral_constant<int, L>(), integral_constant<int, N / V>());
        GS_SHAPE(false_type, 8, 2) GS_SHAPE(false_type, 8, 3) GS_SHAPE(false_type, 8, 4)
        GS_SHAPE(false_type, 8, 6) GS_SHAPE(false_type, 16, 4) GS_SHAPE(false_type, 16, 6)
        GS_SHAPE(false_type, 32, 4) GS_SHAPE(false_type, 32, 5)
        GS_SHAPE(true_type, 32, 6) GS_SHAPE(true_type, 32, 8) GS_SHAPE(true_type, 64, 6)
        GS_SHAPE(true_type, 64, 8) GS_SHAPE(true_type, 128, 6) GS_SHAPE(true_type, 128, 8)
        GS_SHAPE(true_type, 256, 6) GS_SHAPE(true_type, 256, 8) GS_SHAPE(true_type, 512, 6)
#undef GS_SHAPE
    } else {
        const int runs = (D + V - 1) / V;
        if (runs <= 4) return f(false_type(), integral_constant<int, 4>(), integral_constant<int, 1>());
        if (runs <= 8) return f(false_type(), integral_constant<int, 8>(), integral_constant<int, 1>());
        if (runs <= 16) return f(false_type(), integral_constant<int, 16>(), integral_constant<int, 1>());
        if (runs <= 32) return f(false_type(), integral_constant<int, 32>(), integral_constant<int, 1>());
        if constexpr (V == 4)   // of eight elements, 32 runs are 256
            if (D <= 256) return f(true_type(), integral_constant<int, 32>(), integral_constant<int, NV>());
        if (D <= 512) return f(true_type(), integral_constant<int, 64>(), integral_constant<int, NV>());
        if (D <= 1024) return f(true_type(), integral_constant<int, 128>(), integral_constant<int, NV>());
        if (D <= 2048) return f(true_type(), integral_constant<int, 256>(), integral_constant<int, NV>());
    }
    if (D <= kResStaged) return f(true_type(), integral_constant<int, 512>(), integral_constant<int, NV>());
    if constexpr (!MORE) return f(false_type(), integral_constant<int, 512>(), integral_constant<int, 2 * NV>());
    return cudaErrorInvalidValue;   // not reached: rows that are read again
}
// Rows that are read again for the sums: those that do not fit a block's registers beside
// more than two sums (2048 x 8192 bf16: two sums in registers 45 us, read again 84; five
// 129 and 88; 4088 x 4104 fp32 77 and 126; 358 and 142).
inline bool resnorm_wide(const ResNormArgs &a, bool post) {
    return a.D > kResOnChip || (a.D > kResStaged && (post || a.groups > 0));
}

template <typename T, int V> ResNormPlan resnorm_plan_of(const ResNormArgs &a, bool post) {
    ResNormPlan q = {};
    if (resnorm_wide(a, post)) {
        const int columns = resnorm_sums_columns(a.D, V);
        return resnorm_plan(a, 1, std::max(1, kResSumsBlocks<V> * kResSms / columns));
    }
    resnorm_backward_shape<V, false>(a.D, [&](auto staged, auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        q = decltype(staged)::value
                ? resnorm_plan(a, kStagedThreads / L, kResSms)
                : resnorm_plan(a, res_block(L) / L, kResSms * resnorm_backward_blocks(L, NV * V));
        return cudaSuccess;
    });
    return q;
}

// Workspace: the blocks' column sums, the segments' sums for the gate, and the means
// of rows wider than kResStaged.
struct ResNormLayout {
    size_t gate, means, bytes;
    ResNormLayout(const ResNormArgs &a, const ResNormPlan &q, bool post) {
        const bool wide = resnorm_wide(a, post);
        const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
        gate = up((size_t)q.blocks * 4 * a.D * sizeof(float));
        // one gate: a row of sums per block, but per chunk for wide rows
        const size_t sums = a.groups == 0                        ? 0
                            : a.groups == 1 && !wide             ? q.blocks
                            : q.chunks > 1                       ? (size_t)q.groups * q.chunks
                                                                 : 0;
        means = gate + up(sums * a.D * sizeof(float));
        bytes = means + (wide ? up((size_t)a.rows * sizeof(float2)) : 0);
    }
};

template <typename T> size_t resnorm_ws_bytes(const ResNormArgs &a) {
    size_t most = 0;   // whatever the alignment will be, with z_scale or without
    for (const bool post : {false, true}) {
        most = std::max(most, ResNormLayout(a, resnorm_plan_of<T, 1>(a, post), post).bytes);
        most = std::max(most, ResNormLayout(a, resnorm_plan_of<T, 2>(a, post), post).bytes);
        most = std::max(most, ResNormLayout(a, resnorm_plan_of<T, kVec<T>>(a, post), post).bytes);
    }
    return most;
}

// Calls f(V) with the elements of a run: 16 bytes, 2 or 1, as the width and the addresses
// allow (21788 x 770 bf16 by pairs 42 us, by single elements 63; backward 78 and 96).
template <typename T, typename F>
auto resnorm_width(int D, std::initializer_list<const void *> tensors, F &&f) {
    uintptr_t all = (uintptr_t)D * sizeof(T);
    for (const void *t : tensors) all |= (uintptr_t)t;
    if (all % 16 == 0) return f(std::integral_constant<int, kVec<T>>());
    if (all % (2 * sizeof(T)) == 0) return f(std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>());
}

template <typename T, int V>
cudaError_t run_resnorm(const ResNormArgs &a, const ResNormPtrs &p, cudaStream_t s) {
    return resnorm_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        // (two rows per team 69.5 us for 524288 x 64 bf16, one 63)
        constexpr int kRows = res_block(L) / L;
        const auto kernel = p.z_scale ? resnorm_kernel<T, V, L, NV, true>
                                      : resnorm_kernel<T, V, L, NV, false>;
        kernel<<<(unsigned)((a.rows + kRows - 1) / kRows), res_block(L), 0, s>>>(a, p);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t launch_resnorm(const ResNormArgs &a, const ResNormPtrs &p, cudaStream_t s) {
    return resnorm_width<T>(
        a.D, {p.X, p.Z, p.gate, p.z_scale, p.z_B, p.scale, p.B, p.S, p.Y}, [&](auto v) {
            constexpr int V = decltype(v)::value;
            if (a.D <= kResOnChip) return run_resnorm<T, V>(a, p, s);
            if (sizeof(T) == 4 || resnorm_large<T>(a)) {   // in fp32 they all are
                resnorm_wide_kernel<T, V, 512><<<(unsigned)a.rows, 512, 0, s>>>(a, p);
            } else if constexpr (sizeof(T) == 2) {
                resnorm_wide_kernel<T, V, 256><<<(unsigned)a.rows, 256, 0, s>>>(a, p);
            }
            return cudaGetLastError();
        });
}

template <typename T, int V, int L, int NV, bool POST, bool GATE>
cudaError_t run_resnorm_staged(const ResNormArgs &a, const ResNormPtrs &p, const ResNormPlan &q,
                               float *partials, float *gate_partials, cudaStream_t s) {
    static_assert(staged_shape(L * kStagedN, sizeof(T), L, POST, GATE, true).stages >= 2,
                  "a row being worked on and one ahead");
    const auto kernel = resnorm_staged_kernel<T, V, L, NV, POST, GATE>;
    const StagedShape shape = staged_shape(a.D, sizeof(T), L, POST, GATE, p.dS);
    const int rows = kStagedThreads / L * shape.stages * (shape.arrays * shape.pitch + kStagedStats);
    const int join = kStagedThreads > L ? kStagedThreads * kStagedN * (int)sizeof(float) : 0;
    const int smem = 4 * staged_totals(POST, GATE) + std::max(rows, join);
    static DeviceFlags ready;
    const cudaError_t e = once_per_device(ready, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedRing);
    });
    if (e != cudaSuccess) return e;
    kernel<<<q.blocks, kStagedThreads, smem, s>>>(a, p, q, shape, partials, gate_partials);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_resnorm_backward(const ResNormArgs &a, const ResNormPtrs &p, const ResNormPlan &q,
                                 float *partials, float *gate_partials, cudaStream_t s) {
    const auto form = [&](auto post, auto gate) {
        constexpr bool POST = decltype(post)::value, GATE = decltype(gate)::value;
        return resnorm_backward_shape<V, POST || GATE>(a.D, [&](auto staged, auto l, auto nv) {
            constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
            if constexpr (decltype(staged)::value) {
                return run_resnorm_staged<T, V, L, NV, POST, GATE>(a, p, q, partials, gate_partials, s);
            } else {
                resnorm_backward_kernel<T, V, L, NV, POST, GATE>
                    <<<q.blocks, res_block(L), 0, s>>>(a, p, q, partials, gate_partials);
                return cudaGetLastError();
            }
        });
    };
    using std::false_type;
    using std::true_type;
    if (p.z_scale) return a.groups > 0 ? form(true_type(), true_type()) : form(true_type(), false_type());
    return a.groups > 0 ? form(false_type(), true_type()) : form(false_type(), false_type());
}

// Rows wider than kResStaged.
template <typename T, int V>
cudaError_t run_resnorm_wide(const ResNormArgs &a, const ResNormPtrs &p, const ResNormPlan &q,
                             float2 *means, float *partials, float *gate_partials, cudaStream_t s) {
    const bool large = resnorm_large<T>(a);
    const auto kernel = large ? resnorm_wide_backward_kernel<T, V, 512> : resnorm_wide_backward_kernel<T, V, 256>;
    kernel<<<(unsigned)a.rows, large ? 512 : 256, 0, s>>>(a, p, means);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!partials && a.groups == 0)) return e;
    return launch_next(true, resnorm_wide_sums_kernel<T, V>,
                       dim3(resnorm_sums_columns(a.D, V), q.blocks), kResThreads, 0, s, a, p, q, means,
                       partials, gate_partials);
}

template <typename T>
cudaError_t launch_resnorm_backward(const ResNormArgs &a, const ResNormPtrs &p, void *ws,
                                    cudaStream_t s) {
    const bool sums = p.dScale || p.dB || p.dz_scale || p.dz_B;
    const bool wide = resnorm_wide(a, p.z_scale);
    ResNormPlan q = {};
    SumArgs sum = {};
    if (a.rows > 0) {
        const cudaError_t e = resnorm_width<T>(
            a.D,
            {p.dS, p.dY, p.S, p.Z, p.gate, p.z_scale, p.z_B, p.scale, p.dX, p.dZ, p.dgate},
            [&](auto v) {
                constexpr int V = decltype(v)::value;
                q = resnorm_plan_of<T, V>(a, p.z_scale);
                const ResNormLayout at(a, q, p.z_scale);
                char *base = (char *)ws;
                float *partials = sums ? (float *)base : nullptr, *gates = (float *)(base + at.gate);
                sum.from = partials;
                sum.group_from = gates;
                return wide ? run_resnorm_wide<T, V>(a, p, q, (float2 *)(base + at.means), partials,
                                                     gates, s)
                            : run_resnorm_backward<T, V>(a, p, q, partials, gates, s);
            });
        if (e != cudaSuccess) return e;
        const bool by_block = a.groups == 1 && !wide;
        if (by_block || (a.groups > 0 && q.chunks > 1)) {
            sum.group_to = p.dgate;
            sum.groups = a.groups;
            sum.group_count = by_block ? q.blocks : q.chunks;
        }
    }
    // without rows the sums are zeros
    sum.vectors = !sums ? 0 : p.z_scale ? 4 : 2;
    sum.count = q.blocks;
    sum.pitch = (int64_t)sum.vectors * a.D;
    sum.to[0] = p.dScale;
    sum.to[1] = p.dB;
    sum.to[2] = p.dz_scale;
    sum.to[3] = p.dz_B;
    sum.D = a.D;
    return launch_sums<T>(sum, a.rows > 0, s);
}

// The gradient by single elements and by pairs is compiled by itself.
#define GS_RESNORM_BACKWARD(T, V)                                                                \
    template cudaError_t run_resnorm_backward<T, V>(const ResNormArgs &, const ResNormPtrs &,     \
                                                    const ResNormPlan &, float *, float *,        \
                                                    cudaStream_t);

#define GS_RESNORM_INST(T)                                                                       \
    extern GS_RESNORM_BACKWARD(T, 1)                                                              \
    extern GS_RESNORM_BACKWARD(T, 2)                                                              \
    template size_t resnorm_ws_bytes<T>(const ResNormArgs &);                                     \
    template cudaError_t launch_resnorm<T>(const ResNormArgs &, const ResNormPtrs &, cudaStream_t); \
    template cudaError_t launch_resnorm_backward<T>(const ResNormArgs &, const ResNormPtrs &,     \
                                                    void *, cudaStream_t);

}  // namespace gs
