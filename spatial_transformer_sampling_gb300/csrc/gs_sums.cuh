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

// 32 columns a block (x), a vector per y: 32 threads per column with every 32nd row
// each, joined in order.
template <typename T> __global__ void __launch_bounds__(1024) sum_rows_kernel(SumArgs a) {
    __shared__ float s[32][33];
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
        for (int b = slice; b < count; b += 32) sum += __ldg(in + b * pitch + d);
    }
    s[slice][lane] = sum;
    __syncthreads();
    // a warp per column: lane `lane` holds slice `lane` of column `slice`
    float v = s[lane][slice];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 32 + slice < a.D) out[blockIdx.x * 32 + slice] = IO<T>::st(v);
}

template <typename T>
cudaError_t launch_sums(const SumArgs &a, bool follows, cudaStream_t s) {
    const int vectors = a.vectors + a.groups;
    if (vectors == 0) return cudaSuccess;
    return launch_next(follows, sum_rows_kernel<T>, dim3((a.D + 31) / 32, vectors), 1024, 0, s, a);
}

}  // namespace gs
