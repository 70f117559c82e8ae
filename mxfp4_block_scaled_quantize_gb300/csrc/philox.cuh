// philox.cuh -- the random bits of every stochastic rounding: Philox4x32-10 (Salmon, Moraes, Dror,
// Shaw, SC 2011), a function of a 128-bit counter and a 64-bit key, so that an element's bits
// depend on its place and the caller's seed alone.
#pragma once

#include <cstdint>

namespace mxfp4 {

__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint64_t seed) {
    uint32_t x0 = c0, x1 = c1, x2 = c2, x3 = c3;
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int round = 0; round < 10; ++round) {
        uint64_t p0, p1;   // full 64-bit products, one wide multiply each
        asm("mul.wide.u32 %0, %1, 0xD2511F53;" : "=l"(p0) : "r"(x0));
        asm("mul.wide.u32 %0, %1, 0xCD9E8D57;" : "=l"(p1) : "r"(x2));
        const uint32_t hi0 = static_cast<uint32_t>(p0 >> 32), lo0 = static_cast<uint32_t>(p0);
        const uint32_t hi1 = static_cast<uint32_t>(p1 >> 32), lo1 = static_cast<uint32_t>(p1);
        const uint32_t n0 = hi1 ^ x1 ^ k0, n2 = hi0 ^ x3 ^ k1;
        x0 = n0;
        x1 = lo1;
        x2 = n2;
        x3 = lo0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

__device__ __forceinline__ uint4 philox4x32_10(uint32_t c0, uint32_t c1, uint32_t c2, uint64_t seed) {
    return philox4x32_10(c0, c1, c2, 0u, seed);
}

}  // namespace mxfp4
