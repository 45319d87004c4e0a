// gs_vec.cuh -- runs of V consecutive elements moved in one access (16 bytes,
// or a single element where rows or bases are not 16-byte aligned), widened to
// fp32.
#pragma once

#include "gs_common.cuh"

namespace gs {

template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

template <typename T, int V> struct Run {
    static_assert(V == 1 || V * sizeof(T) == 16, "a run is one element or 16 bytes");
    using Raw = std::conditional_t<V == 1, T, uint4>;
    static __device__ __forceinline__ Raw load(const T *p) {
        return *reinterpret_cast<const Raw *>(p);
    }
    static __device__ __forceinline__ Raw zero() { return Raw(); }
    static __device__ __forceinline__ void widen(const Raw &r, float (&v)[V]) {
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = IO<T>::to_f(e[k]);
    }
    static __device__ __forceinline__ void store(T *p, const float (&v)[V]) {
        Raw r;
        T *e = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int k = 0; k < V; ++k) e[k] = IO<T>::st(v[k]);
        *reinterpret_cast<Raw *>(p) = r;
    }
};

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace gs
