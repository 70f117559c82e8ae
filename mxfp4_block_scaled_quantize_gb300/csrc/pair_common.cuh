// pair_common.cuh -- what the CTA-pair MXF4 kernels share: the instruction descriptor of the
// 256-row block-scaled MMA, and the swizzled shared-memory staging of an epilogue warp's
// 32-row x 64-byte output piece.
#pragma once

#include <cstdint>

namespace mxfp4 {

constexpr int kOutRowBytes = 64;
constexpr int kOutBytes = 32 * kOutRowBytes;

// tcgen05.mma kind::mxf4 instruction descriptor, M = 256 (the pair), N = n.
__device__ __forceinline__ uint32_t pair_idesc(uint32_t sf_id, uint32_t n) {
    uint32_t d = 0;
    d |= sf_id << 4;
    d |= 1u << 7;
    d |= 1u << 10;
    d |= (n >> 3) << 17;
    d |= 1u << 23;
    d |= static_cast<uint32_t>(256 >> 4) << 24;
    d |= sf_id << 29;
    return d;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ uint32_t swz64(uint32_t r, uint32_t j) {
    return r * kOutRowBytes + ((j ^ ((r >> 1) & 3u)) << 4);
}

}  // namespace mxfp4
