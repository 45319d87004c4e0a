// gs_philox.cuh -- the Philox4x32-10 counter-based generator (Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011): ten
// rounds of two 32 x 32 -> 64 bit products, exclusive-or with the key and a
// fixed word permutation; the key advances by a Weyl step per round.
#pragma once

#include <stdint.h>

namespace gs {

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;

// Key of every round, for (lo, hi) words of `key`.
struct PhiloxKeys {
    uint32_t k0[10], k1[10];
};
inline PhiloxKeys philox_keys(uint64_t key) {
    PhiloxKeys k;
    for (int r = 0; r < 10; ++r) {
        k.k0[r] = (uint32_t)key + (uint32_t)r * 0x9E3779B9u;
        k.k1[r] = (uint32_t)(key >> 32) + (uint32_t)r * 0xBB67AE85u;
    }
    return k;
}

// The four words of counter {low, high, stream lo, stream hi}.  `high` and
// `stream` are the same for a whole block, so that the first round's second
// product and the second round's first one are computed once per block (the
// compiler keeps them in uniform registers).
__device__ __forceinline__ void philox4x32_10(uint32_t low, uint32_t high, uint64_t stream,
                                              const PhiloxKeys &keys, uint32_t (&w)[4]) {
    uint32_t c0 = low, c1 = high, c2 = (uint32_t)stream, c3 = (uint32_t)(stream >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)c0 * kPhiloxM0, p1 = (uint64_t)c2 * kPhiloxM1;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ keys.k0[r];
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ keys.k1[r];
        c3 = (uint32_t)p0;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
}

}  // namespace gs
