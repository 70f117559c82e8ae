// norm_row.cuh -- what the layer norm's passes share: a thread's part of a row, and sums over a row.
#pragma once

#include <cuda_bf16.h>

#include "launch_norm.h"
#include "ptx.cuh"

namespace mxfp4 {

// A thread's 8 kGroups elements of a row.  kWide: groups of 8 consecutive elements, one or two 16-byte
// accesses each (pitches and dim are multiples of 8 and every address of 16 bytes); else elements
// `threads` apart, one by one.  Threads past the row hold zeros.
template <bool kF32, bool kWide, int kGroups>
struct RowPart {
    static constexpr int kElements = 8 * kGroups;
    static constexpr int kWords = kElements / (kF32 ? 1 : 2);
    uint32_t w[kWords];

    __device__ __forceinline__ static int column(int k, int t, int threads) {
        return kWide ? ((k >> 3) * threads + t) * 8 + (k & 7) : k * threads + t;
    }
    __device__ __forceinline__ void load(const void* row, int dim, int t, int threads) {
        if (kWide) {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const int c = (j * threads + t) * 8;
                constexpr int kLoads = kF32 ? 2 : 1;
#pragma unroll
                for (int h = 0; h < kLoads; ++h) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (c < dim) v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(row) + static_cast<int64_t>(c) * (kF32 ? 4 : 2))[h];
                    uint32_t* const d = w + (j * kLoads + h) * 4;
                    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[k] = 0u;
#pragma unroll
            for (int k = 0; k < kElements; ++k) {
                const int c = k * threads + t;
                if (c >= dim) continue;
                if (kF32) w[k] = static_cast<const uint32_t*>(row)[c];
                else w[k >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[c]) << (16 * (k & 1));
            }
        }
    }
    __device__ __forceinline__ float get(int k) const {
        if (kF32) return __uint_as_float(w[k]);
        return __uint_as_float(k & 1 ? w[k >> 1] & 0xFFFF0000u : w[k >> 1] << 16);
    }
    // f[k] for the elements of the row, rounded once to its type.
    __device__ __forceinline__ static void store(void* row, const float* f, int dim, int t, int threads) {
        if (kWide) {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const int c = (j * threads + t) * 8;
                if (c >= dim) continue;
                if (kF32) {
                    float4* const d = reinterpret_cast<float4*>(static_cast<float*>(row) + c);
                    d[0] = make_float4(f[8 * j], f[8 * j + 1], f[8 * j + 2], f[8 * j + 3]);
                    d[1] = make_float4(f[8 * j + 4], f[8 * j + 5], f[8 * j + 6], f[8 * j + 7]);
                } else {
                    uint32_t v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(f[8 * j + 2 * i], f[8 * j + 2 * i + 1]);
                        v[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + c) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kElements; ++k) {
                const int c = k * threads + t;
                if (c >= dim) continue;
                if (kF32) static_cast<float*>(row)[c] = f[k];
                else static_cast<__nv_bfloat16*>(row)[c] = __float2bfloat16_rn(f[k]);
            }
        }
    }
};

// A thread's part of a vector of fp32 or bf16, as floats, `past` behind the row's end.
template <bool kWide, int kGroups>
__device__ __forceinline__ void load_vector(const void* v, int64_t at, bool f32, int dim, int t, int threads, float* f) {
    if (f32) {
        RowPart<true, kWide, kGroups> p;
        p.load(static_cast<const float*>(v) + at, dim, t, threads);
#pragma unroll
        for (int k = 0; k < 8 * kGroups; ++k) f[k] = p.get(k);
    } else {
        RowPart<false, kWide, kGroups> p;
        p.load(static_cast<const uint16_t*>(v) + at, dim, t, threads);
#pragma unroll
        for (int k = 0; k < 8 * kGroups; ++k) f[k] = p.get(k);
    }
}

__device__ __forceinline__ float2 warp_sum2(float2 v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, d);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, d);
    }
    return v;
}

// Two sums over the row's threads, in all of them and in the same order in each.  A row of several
// warps goes through `shared` ([32] of its own for each of two calls in a row: one barrier a call).
template <bool kWarpRow>
__device__ __forceinline__ float2 row_sum2(float2 v, float2* shared) {
    v = warp_sum2(v);
    if (kWarpRow) return v;
    const int warps = blockDim.x >> 5;
    if (lane_id() == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = static_cast<int>(lane_id()) < warps ? shared[lane_id()] : make_float2(0.0f, 0.0f);
    return warp_sum2(v);
}

}  // namespace mxfp4
