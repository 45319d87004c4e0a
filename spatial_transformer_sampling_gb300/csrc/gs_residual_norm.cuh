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
// share it, NV runs of V elements each, up to D = 8192; longer rows are read again
// for each pass.  Backward, each team of L threads walks segments: rows that share a
// gate, or every chunks-th of them.  A thread keeps the sums of its columns over all
// its rows, and those for the gate over a segment; a second kernel adds the teams'
// sums in order.
#pragma once

#include "gs_sums.cuh"

namespace gs {

constexpr int kResThreads = 256;       // of a block, at least
constexpr int kResOnChip = 8192;       // widest row held in registers
constexpr int kResSms = 152;
constexpr int kResWideBlocks = 2;      // of the column sums of wider rows, per SM

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

// R rows per team of L threads, loads of all of them first.
template <typename T, int V, int L, int NV, int R, bool POST>
__global__ void __launch_bounds__(res_block(L)) resnorm_kernel(ResNormArgs a, ResNormPtrs p) {
    using IOV = Run<T, V>;
    constexpr int kTeams = res_block(L) / L;
    const int part = threadIdx.x % L;
    const int64_t row0 = ((int64_t)blockIdx.x * kTeams + threadIdx.x / L) * R;
    const float per_d = 1.0f / (float)a.D;
    typename IOV::Raw rx[R][NV], rz[R][NV], rg[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = row0 + r;
        const int64_t gate = a.groups > 0 && row < a.rows ? row / a.group_rows * a.D : 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = row < a.rows && d < a.D;
            rx[r][k] = on ? IOV::load((const T *)p.X + row * a.D + d) : IOV::zero();
            rz[r][k] = on ? IOV::load((const T *)p.Z + row * a.D + d) : IOV::zero();
            if (a.groups > 0) rg[r][k] = on ? IOV::load((const T *)p.gate + gate + d) : IOV::zero();
        }
    }
    int slot = 0;
    // v minus its mean, and the mean and reciprocal deviation
    const auto normalise = [&](float (&v)[NV][V], float &mean, float &inv) {
        mean = 0.0f;
        if (a.layer) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) s += v[k][e];
            mean = team_sum<L>(s, slot) * per_d;
        }
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const float m = (k * L + part) * V < a.D ? mean : 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[k][e] -= m;
                s = fmaf(v[k][e], v[k][e], s);
            }
        }
        inv = 1.0f / sqrtf(fmaf(team_sum<L>(s, slot), per_d, a.eps));
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = row0 + r;
        float v[NV][V];
        float4 stats = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k) IOV::widen(rz[r][k], v[k]);
        if (POST) normalise(v, stats.x, stats.y);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            const bool on = d < a.D;
            if (POST) {
                float w[V], b[V] = {};
                IOV::widen(on ? IOV::load((const T *)p.z_scale + d) : IOV::zero(), w);
                if (p.z_B) IOV::widen(on ? IOV::load((const T *)p.z_B + d) : IOV::zero(), b);
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = on ? fmaf(v[k][e] * stats.y, w[e], b[e]) : 0.0f;
            }
            float x[V], g[V];
            IOV::widen(rx[r][k], x);
            if (a.groups > 0) {
                IOV::widen(rg[r][k], g);
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = fmaf(g[e], v[k][e], a.alpha * x[e]);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) v[k][e] = fmaf(a.alpha, x[e], v[k][e]);
            }
            if (row < a.rows && on) IOV::store((T *)p.S + row * a.D + d, v[k]);
        }
        normalise(v, stats.z, stats.w);
        if (row >= a.rows) continue;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int d = (k * L + part) * V;
            if (d >= a.D) continue;
            float w[V], b[V] = {}, y[V];
            IOV::widen(IOV::load((const T *)p.scale + d), w);
            if (p.B) IOV::widen(IOV::load((const T *)p.B + d), b);
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = fmaf(v[k][e] * stats.w, w[e], b[e]);
            IOV::store((T *)p.Y + row * a.D + d, y);
        }
        if (part == 0 && p.stats) *reinterpret_cast<float4 *>(p.stats + 4 * row) = stats;
    }
}

// Rows wider than kResOnChip: a block per row that reads it again for each sum.
template <typename T>
__global__ void __launch_bounds__(kResThreads) resnorm_wide_kernel(ResNormArgs a, ResNormPtrs p) {
    const int64_t row = blockIdx.x, at = row * a.D;
    const T *x = (const T *)p.X + at, *z = (const T *)p.Z + at;
    const T *gate = a.groups > 0 ? (const T *)p.gate + row / a.group_rows * a.D : nullptr;
    const float per_d = 1.0f / (float)a.D;
    int slot = 0;
    const auto statistics = [&](auto value, float &mean, float &inv) {
        float s = 0.0f;
        mean = 0.0f;
        if (a.layer) {
            for (int d = threadIdx.x; d < a.D; d += kResThreads) s += value(d);
            mean = team_sum<kResThreads>(s, slot) * per_d;
        }
        s = 0.0f;
        for (int d = threadIdx.x; d < a.D; d += kResThreads) {
            const float c = value(d) - mean;
            s = fmaf(c, c, s);
        }
        inv = 1.0f / sqrtf(fmaf(team_sum<kResThreads>(s, slot), per_d, a.eps));
    };
    float4 st = make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    if (p.z_scale) statistics([&](int d) { return IO<T>::ld(z + d); }, st.x, st.y);
    const auto sum = [&](int d) {
        float v = IO<T>::ld(z + d);
        if (p.z_scale)
            v = fmaf((v - st.x) * st.y, IO<T>::ld((const T *)p.z_scale + d),
                     p.z_B ? IO<T>::ld((const T *)p.z_B + d) : 0.0f);
        const float r = IO<T>::ld(x + d);
        return gate ? fmaf(IO<T>::ld(gate + d), v, a.alpha * r) : fmaf(a.alpha, r, v);
    };
    statistics(sum, st.z, st.w);
    for (int d = threadIdx.x; d < a.D; d += kResThreads) {
        const float s = sum(d), b = p.B ? IO<T>::ld((const T *)p.B + d) : 0.0f;
        ((T *)p.S)[at + d] = IO<T>::st(s);
        ((T *)p.Y)[at + d] = IO<T>::st(fmaf((s - st.z) * st.w, IO<T>::ld((const T *)p.scale + d), b));
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
    int64_t segment, row, end, gate;
    int step;
    __device__ __forceinline__ void start(const ResNormPlan &q, int64_t s) {
        segment = s;
        step = 0;
        gate = s / q.chunks;
        const int64_t within = s - gate * q.chunks;
        row = gate < q.groups && within < q.group_rows ? gate * q.group_rows + within : -1;
        end = (gate + 1) * q.group_rows;
    }
    __device__ __forceinline__ void next(const ResNormPlan &q) {
        if (++step < q.steps) {
            if (row >= 0) row += q.chunks;
            if (row >= end) row = -1;
        } else {
            start(q, segment + q.teams);
        }
    }
};

// Blocks per SM, by the elements of a row that a thread holds.
constexpr int resnorm_backward_blocks(int L, int N) {
    return L > kResThreads ? 1 : N <= 4 ? 3 : N <= 8 ? 2 : 1;
}

// dX, dZ and, into partials[block][vector], the block's column sums (for dScale, dB
// and, with POST, dz_scale and dz_B); into gate_partials[segment] those for the gate.
// The next row's loads are issued before this one is worked on.
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
        const int64_t row = w.row, at = row * a.D, gate = w.gate * a.D;
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
    w.start(q, (int64_t)blockIdx.x * kTeams + team);
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
        if (GATE && ends) {
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
    if (!partials) return;
    // the teams of the block in order, one vector and run at a time
    float *out = partials + (int64_t)blockIdx.x * kVectors * a.D;
    __shared__ float join[kTeams > 1 ? kThreads * V : 1];
#pragma unroll
    for (int j = 0; j < kVectors; ++j)
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (kTeams > 1) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < V; ++e) join[threadIdx.x * V + e] = sum[j][k][e];
                __syncthreads();
                for (int c = threadIdx.x; c < L * V; c += kThreads) {
                    const int d = k * L * V + c;
                    float t = 0.0f;
#pragma unroll
                    for (int g = 0; g < kTeams; ++g) t += join[g * L * V + c];
                    if (d < a.D) out[(int64_t)j * a.D + d] = t;
                }
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const int d = (k * L + part) * V + e;
                    if (d < a.D) out[(int64_t)j * a.D + d] = sum[j][k][e];
                }
            }
        }
}

// Rows wider than kResOnChip: a block per row for dX and dZ, which leaves the row's
// two means in `means`; then a thread per column for the sums.
template <typename T>
__global__ void __launch_bounds__(kResThreads)
    resnorm_wide_backward_kernel(ResNormArgs a, ResNormPtrs p, float2 *means) {
    const int64_t row = blockIdx.x, at = row * a.D;
    const T *dS = p.dS ? (const T *)p.dS + at : nullptr, *dY = (const T *)p.dY + at;
    const T *S = (const T *)p.S + at, *Z = (const T *)p.Z + at;
    const T *gate = a.groups > 0 ? (const T *)p.gate + row / a.group_rows * a.D : nullptr;
    const float4 st = __ldg(reinterpret_cast<const float4 *>(p.stats) + row);
    const float per_d = 1.0f / (float)a.D;
    int slot = 0;
    float t0 = 0.0f, t1 = 0.0f;
    for (int d = threadIdx.x; d < a.D; d += kResThreads) {
        const float w = IO<T>::ld(dY + d) * IO<T>::ld((const T *)p.scale + d);
        t0 += w;
        t1 = fmaf(w, (IO<T>::ld(S + d) - st.z) * st.w, t1);
    }
    team_sum2<kResThreads>(t0, t1, slot);
    t0 = a.layer ? t0 * -per_d : 0.0f;
    t1 *= -per_d;
    if (threadIdx.x == 0) means[row] = make_float2(t0, t1);
    const auto ds_of = [&](int d) {
        const float w = IO<T>::ld(dY + d) * IO<T>::ld((const T *)p.scale + d);
        const float sh = (IO<T>::ld(S + d) - st.z) * st.w;
        return fmaf(fmaf(sh, t1, w + t0), st.w, dS ? IO<T>::ld(dS + d) : 0.0f);
    };
    const auto to_z = [&](int d) {
        float v = ds_of(d);
        if (gate) v *= IO<T>::ld(gate + d);
        return p.z_scale ? v * IO<T>::ld((const T *)p.z_scale + d) : v;
    };
    float u0 = 0.0f, u1 = 0.0f;
    for (int d = threadIdx.x; d < a.D; d += kResThreads) {
        ((T *)p.dX)[at + d] = IO<T>::st(a.alpha * ds_of(d));
        const float v = to_z(d);
        if (p.z_scale) {
            u0 += v;
            u1 = fmaf(v, (IO<T>::ld(Z + d) - st.x) * st.y, u1);
        } else {
            ((T *)p.dZ)[at + d] = IO<T>::st(v);
        }
    }
    if (!p.z_scale) return;
    team_sum2<kResThreads>(u0, u1, slot);
    u0 = a.layer ? u0 * -per_d : 0.0f;
    u1 *= -per_d;
    for (int d = threadIdx.x; d < a.D; d += kResThreads)
        ((T *)p.dZ)[at + d] =
            IO<T>::st(fmaf((IO<T>::ld(Z + d) - st.x) * st.y, u1, to_z(d) + u0) * st.y);
}
template <typename T>
__global__ void __launch_bounds__(kResThreads)
    resnorm_wide_sums_kernel(ResNormArgs a, ResNormPtrs p, ResNormPlan q, const float2 *means,
                             float *partials, float *gate_partials) {
    wait_for_previous_kernel(means);
    const int d = blockIdx.x * kResThreads + threadIdx.x;
    if (d >= a.D) return;
    const float scale = IO<T>::ld((const T *)p.scale + d);
    const float zs = p.z_scale ? IO<T>::ld((const T *)p.z_scale + d) : 1.0f;
    const float zb = p.z_B ? IO<T>::ld((const T *)p.z_B + d) : 0.0f;
    float sum[4] = {}, gate_sum = 0.0f;
    ResNormWalk w;
    w.start(q, blockIdx.y);
    for (int64_t n = (int64_t)q.rounds * q.steps; n > 0; --n, w.next(q)) {
        if (w.row >= 0) {
            const int64_t at = w.row * a.D + d;
            const float4 st = __ldg(reinterpret_cast<const float4 *>(p.stats) + w.row);
            const float2 t = __ldg(means + w.row);
            const float y = IO<T>::ld((const T *)p.dY + at);
            const float sh = (IO<T>::ld((const T *)p.S + at) - st.z) * st.w;
            const float zh = (IO<T>::ld((const T *)p.Z + at) - st.x) * st.y;
            float ds = fmaf(fmaf(sh, t.y, y * scale + t.x), st.w,
                            p.dS ? IO<T>::ld((const T *)p.dS + at) : 0.0f);
            sum[0] = fmaf(y, sh, sum[0]);
            sum[1] += y;
            if (a.groups > 0) {
                gate_sum = fmaf(ds, fmaf(zh, zs, zb), gate_sum);
                ds *= IO<T>::ld((const T *)p.gate + w.gate * a.D + d);
            }
            sum[2] = fmaf(ds, zh, sum[2]);
            sum[3] += ds;
        }
        if (a.groups > 0 && w.step + 1 == q.steps) {
            if (w.segment < (int64_t)q.groups * q.chunks) {
                if (q.chunks == 1)
                    ((T *)p.dgate)[w.segment * a.D + d] = IO<T>::st(gate_sum);
                else
                    gate_partials[w.segment * a.D + d] = gate_sum;
            }
            gate_sum = 0.0f;
        }
    }
    if (!partials) return;
    const int vectors = p.z_scale ? 4 : 2;
    for (int j = 0; j < vectors; ++j)
        partials[((int64_t)blockIdx.y * vectors + j) * a.D + d] = sum[j];
}

// Calls f(L, NV) with the threads per row and the runs per thread of the forward
// pass for a row of `runs` runs.
template <int V, typename F> cudaError_t resnorm_shape(int runs, F &&f) {
    using std::integral_constant;
    if (runs <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (runs <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (runs <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (runs <= 64) return f(integral_constant<int, 32>(), integral_constant<int, 2>());
    if (runs <= 128) return f(integral_constant<int, 32>(), integral_constant<int, 4>());
    if (runs <= 256) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (runs <= 512) return f(integral_constant<int, 256>(), integral_constant<int, 2>());
    if (runs <= 1024) return f(integral_constant<int, 256>(), integral_constant<int, 4>());
    if constexpr (V <= 4)
        if (runs <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 8>());
    if constexpr (V == 1)
        return runs <= 4096 ? f(integral_constant<int, 256>(), integral_constant<int, 16>())
                            : f(integral_constant<int, 256>(), integral_constant<int, 32>());
    return cudaErrorInvalidValue;   // not reached: D <= kResOnChip
}

// The same for the backward pass: as many threads per row as keep a thread's share,
// and with it the five sums it holds per element, to one run.
template <int V, typename F> cudaError_t resnorm_backward_shape(int runs, F &&f) {
    using std::integral_constant;
    if (runs <= 8) return f(integral_constant<int, 8>(), integral_constant<int, 1>());
    if (runs <= 16) return f(integral_constant<int, 16>(), integral_constant<int, 1>());
    if (runs <= 32) return f(integral_constant<int, 32>(), integral_constant<int, 1>());
    if (runs <= 64) return f(integral_constant<int, 64>(), integral_constant<int, 1>());
    if (runs <= 128) return f(integral_constant<int, 128>(), integral_constant<int, 1>());
    if (runs <= 256) return f(integral_constant<int, 256>(), integral_constant<int, 1>());
    if (runs <= 512) return f(integral_constant<int, 512>(), integral_constant<int, 1>());
    if (runs <= 1024) return f(integral_constant<int, 512>(), integral_constant<int, 2>());
    if constexpr (V <= 4)
        if (runs <= 2048) return f(integral_constant<int, 512>(), integral_constant<int, 4>());
    if constexpr (V == 1)
        return runs <= 4096 ? f(integral_constant<int, 512>(), integral_constant<int, 8>())
                            : f(integral_constant<int, 512>(), integral_constant<int, 16>());
    return cudaErrorInvalidValue;   // not reached: D <= kResOnChip
}

template <int V> ResNormPlan resnorm_plan_of(const ResNormArgs &a) {
    ResNormPlan q = {};
    if (a.D > kResOnChip) return resnorm_plan(a, 1, kResWideBlocks * kResSms);
    resnorm_backward_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        q = resnorm_plan(a, res_block(L) / L, kResSms * resnorm_backward_blocks(L, NV * V));
        return cudaSuccess;
    });
    return q;
}

// Workspace: the blocks' column sums, the segments' sums for the gate, and the means
// of rows wider than kResOnChip.
struct ResNormLayout {
    size_t gate, means, bytes;
    ResNormLayout(const ResNormArgs &a, const ResNormPlan &q) {
        const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
        gate = up((size_t)q.blocks * 4 * a.D * sizeof(float));
        means = gate + (a.groups > 0 && q.chunks > 1
                            ? up((size_t)q.groups * q.chunks * a.D * sizeof(float))
                            : 0);
        bytes = means + (a.D > kResOnChip ? up((size_t)a.rows * sizeof(float2)) : 0);
    }
};

template <typename T> size_t resnorm_ws_bytes(const ResNormArgs &a) {
    // whatever the alignment will be
    const size_t b1 = ResNormLayout(a, resnorm_plan_of<1>(a)).bytes;
    const size_t bv = ResNormLayout(a, resnorm_plan_of<kVec<T>>(a)).bytes;
    return b1 > bv ? b1 : bv;
}

template <typename T, int V>
cudaError_t run_resnorm(const ResNormArgs &a, const ResNormPtrs &p, cudaStream_t s) {
    return resnorm_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        constexpr int R = L == 256 || NV > 1 ? 1 : 2;
        constexpr int kRows = res_block(L) / L * R;
        const auto kernel = p.z_scale ? resnorm_kernel<T, V, L, NV, R, true>
                                      : resnorm_kernel<T, V, L, NV, R, false>;
        kernel<<<(unsigned)((a.rows + kRows - 1) / kRows), res_block(L), 0, s>>>(a, p);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t launch_resnorm(const ResNormArgs &a, const ResNormPtrs &p, cudaStream_t s) {
    if (a.D > kResOnChip) {
        resnorm_wide_kernel<T><<<(unsigned)a.rows, kResThreads, 0, s>>>(a, p);
        return cudaGetLastError();
    }
    if (a.D % kVec<T> == 0 && aligned16(p.X) && aligned16(p.Z) && aligned16(p.gate) &&
        aligned16(p.z_scale) && aligned16(p.z_B) && aligned16(p.scale) && aligned16(p.B) &&
        aligned16(p.S) && aligned16(p.Y))
        return run_resnorm<T, kVec<T>>(a, p, s);
    return run_resnorm<T, 1>(a, p, s);
}

template <typename T, int V>
cudaError_t run_resnorm_backward(const ResNormArgs &a, const ResNormPtrs &p, const ResNormPlan &q,
                                 float *partials, float *gate_partials, cudaStream_t s) {
    return resnorm_backward_shape<V>((a.D + V - 1) / V, [&](auto l, auto nv) {
        constexpr int L = decltype(l)::value, NV = decltype(nv)::value;
        const bool post = p.z_scale, gate = a.groups > 0;
        const auto kernel = post ? (gate ? resnorm_backward_kernel<T, V, L, NV, true, true>
                                         : resnorm_backward_kernel<T, V, L, NV, true, false>)
                                 : (gate ? resnorm_backward_kernel<T, V, L, NV, false, true>
                                         : resnorm_backward_kernel<T, V, L, NV, false, false>);
        kernel<<<q.blocks, res_block(L), 0, s>>>(a, p, q, partials, gate_partials);
        return cudaGetLastError();
    });
}

template <typename T>
cudaError_t launch_resnorm_backward(const ResNormArgs &a, const ResNormPtrs &p, void *ws,
                                    cudaStream_t s) {
    const bool sums = p.dScale || p.dB || p.dz_scale || p.dz_B;
    const bool wide = a.D > kResOnChip;
    const bool runs = a.D % kVec<T> == 0 && aligned16(p.dS) && aligned16(p.dY) && aligned16(p.S) &&
                      aligned16(p.Z) && aligned16(p.gate) && aligned16(p.z_scale) &&
                      aligned16(p.z_B) && aligned16(p.scale) && aligned16(p.dX) &&
                      aligned16(p.dZ) && aligned16(p.dgate);
    ResNormPlan q = {};
    SumArgs sum = {};
    if (a.rows > 0) {
        q = runs ? resnorm_plan_of<kVec<T>>(a) : resnorm_plan_of<1>(a);
        const ResNormLayout at(a, q);
        char *base = (char *)ws;
        float *partials = sums ? (float *)base : nullptr, *gates = (float *)(base + at.gate);
        cudaError_t e;
        if (wide) {
            float2 *means = (float2 *)(base + at.means);
            resnorm_wide_backward_kernel<T><<<(unsigned)a.rows, kResThreads, 0, s>>>(a, p, means);
            e = cudaGetLastError();
            if (e == cudaSuccess && (sums || a.groups > 0))
                e = launch_next(true, resnorm_wide_sums_kernel<T>,
                                dim3((a.D + kResThreads - 1) / kResThreads, q.blocks), kResThreads, 0,
                                s, a, p, q, means, partials, gates);
        } else {
            e = runs ? run_resnorm_backward<T, kVec<T>>(a, p, q, partials, gates, s)
                     : run_resnorm_backward<T, 1>(a, p, q, partials, gates, s);
        }
        if (e != cudaSuccess) return e;
        sum.from = partials;
        if (a.groups > 0 && q.chunks > 1) {
            sum.group_from = gates;
            sum.group_to = p.dgate;
            sum.groups = a.groups;
            sum.group_count = q.chunks;
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

#define GS_RESNORM_INST(T)                                                                       \
    template size_t resnorm_ws_bytes<T>(const ResNormArgs &);                                     \
    template cudaError_t launch_resnorm<T>(const ResNormArgs &, const ResNormPtrs &, cudaStream_t); \
    template cudaError_t launch_resnorm_backward<T>(const ResNormArgs &, const ResNormPtrs &,     \
                                                    void *, cudaStream_t);

}  // namespace gs
