// Compares the roots and quotients of csrc/adamw_math.cuh with CUDA's rounded intrinsics.
#include <cstdint>
#include <cuda_runtime.h>

#include "adamw_math.cuh"

struct Found {
    unsigned long long checked; // results compared
    unsigned long long bad;     // those that differ
    unsigned long long worst;   // largest difference in ulp
    unsigned long long where;   // bits of one operand that gave a difference (quotients: and of s in the high half)
};

namespace {

__device__ void record(Found* f, uint32_t got, uint32_t want, uint64_t at) {
    if (got == want) return;
    atomicAdd(&f->bad, 1ull);
    const uint32_t d = got > want ? got - want : want - got;
    atomicMax(&f->worst, static_cast<unsigned long long>(d));
    f->where = at;
}

// Every float from bits 0 to `last`, eight to a call; stride: those of a call lie so many apart.
__global__ void roots(Found* f, uint32_t last, uint32_t stride) {
    const uint64_t threads = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    unsigned long long n = 0;
    const uint64_t calls = (last / 8 / stride + 1) * static_cast<uint64_t>(stride);
    for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < calls; t += threads) {
        const uint64_t base = t / stride * stride * 8 + t % stride;
        float v[8], r[8];
        for (int k = 0; k < 8; ++k) {
            const uint64_t b = base + static_cast<uint64_t>(k) * stride;
            v[k] = __uint_as_float(b <= last ? static_cast<uint32_t>(b) : 0u);
            n += b <= last;
        }
        mxfp4::sqrt8(v, r);
        for (int k = 0; k < 8; ++k) record(f, __float_as_uint(r[k]), __float_as_uint(__fsqrt_rn(v[k])), __float_as_uint(v[k]));
    }
    atomicAdd(&f->checked, n);
}

__device__ uint32_t scramble(uint64_t i) {   // some 32 bits of i: a multiplicative mix
    i = (i ^ (i >> 31)) * 0x9E3779B97F4A7C15ull;
    i = (i ^ (i >> 29)) * 0xBF58476D1CE4E5B9ull;
    return static_cast<uint32_t>(i >> 32);
}

// s = 2^se with each of the 2^23 mantissas, x in [2^-xe s, 2^(1 - xe) s) or what 448 s leaves of it,
// `each` mantissas of x for each s.  Below 2^-126 the quotient itself has no full mantissa: left out.
__global__ void quotients(Found* f, int se, int xe, int each) {
    const uint64_t threads = static_cast<uint64_t>(gridDim.x) * blockDim.x;
    unsigned long long n = 0;
    for (uint64_t t = static_cast<uint64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < 1ull << 23; t += threads) {
        const float s = __uint_as_float(static_cast<uint32_t>(se + 127) << 23 | static_cast<uint32_t>(t));
        const float inv = __frcp_rn(s), top = __fmul_ru(s, 448.0f * (1.0f + 0x1p-22f));
        for (int j = 0; j < each; ++j) {
            const float one = __uint_as_float(0x3F800000u | (scramble(t * each + j + 1) & 0x7FFFFFu));
            float x = __fmul_rn(scalbnf(one, -xe), scalbnf(1.0f, se));
            if (j == 0) x = top;
            if (x > top) continue;
            const float want = __fdiv_rn(x, s);
            if (want < 0x1p-126f) continue;
            ++n;
            record(f, __float_as_uint(mxfp4::quotient(x, s, inv)), __float_as_uint(want),
                   static_cast<uint64_t>(__float_as_uint(s)) << 32 | __float_as_uint(x));
        }
    }
    atomicAdd(&f->checked, n);
}

template <typename Launch>
int run(Found* out, Launch launch) {
    Found* f = nullptr;
    if (cudaMalloc(&f, sizeof(Found)) != cudaSuccess) return 1;
    int rc = cudaMemset(f, 0, sizeof(Found)) != cudaSuccess;
    if (rc == 0) {
        launch(f);
        rc = cudaGetLastError() != cudaSuccess || cudaMemcpy(out, f, sizeof(Found), cudaMemcpyDeviceToHost) != cudaSuccess;
    }
    cudaFree(f);
    return rc;
}

}  // namespace

extern "C" int check_roots(Found* out, uint32_t last, uint32_t stride) {
    return run(out, [=](Found* f) { roots<<<152 * 8, 256>>>(f, last, stride); });
}

extern "C" int check_quotients(Found* out, int se, int xe, int each) {
    return run(out, [=](Found* f) { quotients<<<152 * 8, 256>>>(f, se, xe, each); });
}
