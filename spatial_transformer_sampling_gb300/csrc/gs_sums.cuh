// gs_sums.cuh -- column sums that blocks left behind, joined in a fixed order.
#pragma once

#include "gs_internal.h"
#include "gs_ptx.cuh"
#include "gs_vec.cuh"

namespace gs {

// Up to kMostSums output vectors of D elements, each the sum of `count` rows of
// fp32 partials, `pitch` floats apart; and `groups` more vectors, one after another
// in `group_to`, each of `group_count` consecutive rows from group_from on.
constexpr int kMostSums = 4;
struct SumArgs {
    const float *from;
    void *to[kMostSums];
    int vectors, count;
    int64_t pitch;
    const float *group_from;
    void *group_to;
    int groups, group_count;
    int D;
};

// 32 columns a block (x), a vector per y: SLICES threads per column with every
// SLICES-th row each, joined in order.
template <typename T, int SLICES>
__global__ void __launch_bounds__(SLICES * 32) sum_rows_kernel(SumArgs a) {
    __shared__ float s[SLICES][33];
    const int lane = threadIdx.x % 32, slice = threadIdx.x / 32, d = blockIdx.x * 32 + lane;
    const int y = blockIdx.y;
    T *out;
    const float *in;
    int64_t pitch;
    int count;
    if (y < a.vectors) {
        out = (T *)a.to[y];
        in = a.from + (int64_t)y * a.D;
        pitch = a.pitch;
        count = a.count;
    } else {
        const int64_t g = y - a.vectors;
        out = (T *)a.group_to + g * a.D;
        in = a.group_from + g * a.group_count * a.D;
        pitch = a.D;
        count = a.group_count;
    }
    if (y < a.vectors && !out) return;
    float sum = 0.0f;
    wait_for_previous_kernel(in);
    if (d < a.D) {
#pragma unroll 8
        for (int b = slice; b < count; b += SLICES) sum += __ldg(in + b * pitch + d);
    }
    s[slice][lane] = sum;
    __syncthreads();
    if (slice > 0) return;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < SLICES; ++w) v += s[w][lane];
    if (d < a.D) out[d] = IO<T>::st(v);
}

template <typename T>
cudaError_t launch_sums(const SumArgs &a, bool follows, cudaStream_t s) {
    const int vectors = a.vectors + a.groups;
    if (vectors == 0) return cudaSuccess;
    // eight warps a block: 16384 x 1024 rows' sums with sixteen gates 10.7 us with 32
    const dim3 grid((a.D + 31) / 32, vectors);
    return launch_next(follows, sum_rows_kernel<T, 8>, grid, 256, 0, s, a);
}

}  // namespace gs
