// adamw.cu -- one AdamW step (decoupled weight decay) over many tensors in one launch, with
// moments in fp32 or in 8 bits.
//
// Per element, with g the gradient times grad_scale and c = 1 - beta^step:
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2,
//   p = p - lr (m / c1 / (sqrt(v / c2) + eps) + wd p),
// all in fp32; p is the fp32 master where there is one (the bf16 parameter is then its rounding),
// else the parameter itself, rounded once to its type.
//
// 8-bit moments.  A block of 128 consecutive elements shares an fp32 scale, amax / 448 (at least
// 2^-126), and an element is the E4M3 value nearest to it over the scale.  The second moment
// enters p through its square root, and its square spans twice the binades, so what is stored is
// r = sqrt(v): E4M3's 18 binades then hold 36 binades of v.  An r above zero never becomes zero
// (it takes the smallest code): m / sqrt(v) of a small element beside a large one would otherwise
// divide by eps.  An element that is not finite becomes NaN and leaves its block's scale alone.
//
// Rounding of the codes.  To nearest, a code stays where it is as long as a step moves its value
// by less than half a code step, 1/32 to 1/18 of it, relative to its block's largest.  A step
// without gradient takes r to sqrt(beta2) r, which is that far only for beta2 below 0.89: at
// 0.95 a block's small elements follow once their largest moves by itself, and at 0.999 they do
// not follow (gradients 100 times smaller in half of each block left v 7400 times too large
// after 12 000 steps).  So to nearest is for beta2 <= 0.95, and beyond that codes are rounded
// stochastically: to a value's upper neighbour with the probability of its place between the
// two, which makes the expected code the value and each moment's expectation that of its
// recurrence.  What that costs is noise (a pure decay by a factor e has gone through roundings of
// a relative variance of 1/8 at most) and two Philox calls for 8 elements: 280 M elements take
// 934 us, bound by arithmetic, and 695 to nearest; 140 M with fp32 gradients 476 and 405.
//
// Bound by memory: bf16 parameters with masters and bf16 gradients move 28 bytes an element with
// fp32 moments and 16.1 with 8-bit ones.  A thread takes 8 consecutive elements, all of whose
// loads are in flight together; 16 lanes hold a block, so its maxima are four shuffles.  The
// tensor table travels as a kernel parameter: no copy, no allocation, and a graph captures it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstring>

#include "adamw_math.cuh"
#include "launch.h"
#include "launch_adamw.h"
#include "philox.cuh"
#include "ptx.cuh"

namespace mxfp4 {
namespace {

// Threads of a CTA.  With 8-bit moments the arithmetic (some 65 instructions an element) nearly
// fills the time of the memory, and many small CTAs keep both busy: one warp takes 715 us for 280 M
// elements (6.3 TB/s, 0.94 of the measured copy), two 784, four 748.  For 140 M in tensors of odd
// sizes with fp32 gradients it is 424, 458 and 405: there four warps gain what they lose on whole
// tensors, and one warp is kept for both.  With fp32 moments, 69.7 M elements in 48 tensors, 128
// threads take 280.5 us (7.0 TB/s), 64 284 and one warp 288.  (Steps back to back.)
constexpr int kThreads32 = 128;   // fp32 moments
constexpr int kThreads8 = 32;     // 8-bit moments
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126
constexpr double kNearestBeta2 = 0.95;         // largest beta2 with codes to nearest
constexpr float kMinCode = 0.001953125f;       // 2^-9, the smallest E4M3 value above zero

__device__ __forceinline__ void unpack_bf16(const uint4& u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight elements at i: with wide loads where they are whole and aligned, else one by one, zero past n.
template <bool kF32>
__device__ __forceinline__ void load8(const void* p, int64_t i, int64_t n, bool wide, float* f) {
    if (wide) {
        if (kF32) {
            const float4* const s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
            const float4 a = s[0], b = s[1];
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        } else {
            unpack_bf16(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i), f);
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        f[k] = 0.0f;
        if (i + k < n)
            f[k] = kF32 ? static_cast<const float*>(p)[i + k]
                        : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + k]) << 16);
    }
}

template <bool kF32>
__device__ __forceinline__ void store8(void* p, int64_t i, int64_t n, bool wide, const float* f) {
    if (wide) {
        if (kF32) {
            float4* const d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
            d[0] = make_float4(f[0], f[1], f[2], f[3]);
            d[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (i + k >= n) break;
        if (kF32)
            static_cast<float*>(p)[i + k] = f[k];
        else
            static_cast<__nv_bfloat16*>(p)[i + k] = __float2bfloat16_rn(f[k]);
    }
}

__device__ __forceinline__ uint2 load_codes(const void* p, int64_t i, int64_t n, bool wide) {
    const uint8_t* const s = static_cast<const uint8_t*>(p) + i;
    if (wide) return *reinterpret_cast<const uint2*>(s);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k < n) w[k >> 2] |= static_cast<uint32_t>(s[k]) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t n, bool wide, uint2 q) {
    uint8_t* const d = static_cast<uint8_t*>(p) + i;
    if (wide) {
        *reinterpret_cast<uint2*>(d) = q;
        return;
    }
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (i + k < n) d[k] = static_cast<uint8_t>(w[k >> 2] >> (8 * (k & 3)));
}

__device__ __forceinline__ void decode_e4m3(uint2 q, float scale, float* f) {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t h;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(h)
            : "r"(w[k >> 1] >> (16 * (k & 1))));
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * k] = v.x * scale;
        f[2 * k + 1] = v.y * scale;
    }
}

__device__ __forceinline__ uint2 encode_e4m3(const float* f) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        asm("{\n\t.reg .b16 lo, hi;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
            "mov.b32 %0, {lo, hi};\n\t}"
            : "=r"(w[k])
            : "f"(f[4 * k]), "f"(f[4 * k + 1]), "f"(f[4 * k + 2]), "f"(f[4 * k + 3]));
    return make_uint2(w[0], w[1]);
}

// Stochastic rounding onto E4M3's magnitudes (steps of g = 2^(e - 3) in [2^e, 2^(e + 1)), 2^-9
// below 2^-6): a = |y| <= 448 (1 + 2^-22), x: a value with y's sign, r: 16 random bits.  Gives the
// lower neighbour lo unless (a - lo) / g >= (r + 1/2) / 2^16, so that the chance of the upper one
// is its share rounded to 2^-16, not cut off.  As in the MXFP4 quantizer: a + noise, noise =
// g (1 + (65535.5 - r) / 2^16) from bits, rounded toward zero, then onto the multiples of g by
// adding g 2^23 toward zero, and both offsets taken off again.
__device__ __forceinline__ float sr_e4m3(float a, float x, uint32_t r) {
    const uint32_t gbits = (max(__float_as_uint(a) >> 23, 121u) - 3u) << 23;
    const float noise = __uint_as_float(gbits | ((r ^ 0xFFFFu) << 7) | 0x40u);
    const uint32_t cbits = gbits + (23u << 23);
    const float s = __fadd_rz(__fadd_rz(a, noise), __uint_as_float(cbits));
    const float q = __fsub_rn(s, __uint_as_float(cbits + 1u));   // - (g 2^23 + g)
    return __uint_as_float(__float_as_uint(q) | (__float_as_uint(x) & 0x80000000u));
}

// This lane's block (16 lanes) of x: its scale, and the eight codes.  kRoot: values >= 0, of
// which those above zero stay there.  kSr: stochastically, by `bits`, of which element k takes half
// k % 2 of word k / 2.  The quotients x / scale are those of adamw_math.cuh.
template <bool kRoot, bool kSr>
__device__ __forceinline__ uint2 encode_block(const float* x, float* scale, uint4 bits) {
    const float inf = __int_as_float(0x7F800000);
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max_nan(top, fabsf(x[k]));
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const bool odd = !(top < inf);   // the block holds a value that is not finite: rare
    if (__any_sync(0xFFFFFFFFu, odd)) {
        float t = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = fmaxf(t, fabsf(x[k]) < inf ? fabsf(x[k]) : 0.0f);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, d));
        top = t;
    }
    const float s = fmaxf(__fmul_rn(top, 1.0f / kE4m3Max), kMinScale);
    const float inv = __frcp_rn(s);
    *scale = s;
    const uint32_t rnd[4] = {bits.x, bits.y, bits.z, bits.w};
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        y[k] = quotient(x[k], s, inv);
        if (kSr) y[k] = sr_e4m3(fabsf(y[k]), x[k], k & 1 ? rnd[k >> 1] >> 16 : rnd[k >> 1] & 0xFFFFu);
        if (kRoot) y[k] = x[k] > 0.0f ? fmaxf(y[k], kMinCode) : 0.0f;
    }
    if (odd) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (!(fabsf(x[k]) < inf)) y[k] = __int_as_float(0x7FC00000);
    }
    return encode_e4m3(y);
}

struct Hyper {
    float beta1, one_beta1, beta2, one_beta2, eps, step_c1, inv_root_c2, decay, grad_scale;
    uint32_t tensor, step;   // of the random bits' counter
    uint64_t seed;
};

// Eight elements of t at i.  kWhole: all eight exist and every access is aligned.
template <bool kPF32, bool kGF32, bool kState8, bool kSr, bool kWhole>
__device__ __forceinline__ void update8(const mxfp4_adamw_tensor& t, const Hyper& h, int64_t i, int64_t n, bool aligned) {
    // past the end a lane still takes part in its block's maximum, with zeros
    const bool wide = kWhole || (aligned && i + 8 <= n);
    float g[8], p[8], m[8], v[8], r[8];
    load8<kGF32>(t.g, i, n, wide, g);
    if (t.master != nullptr)
        load8<true>(t.master, i, n, wide, p);
    else
        load8<kPF32>(t.p, i, n, wide, p);
    if (kState8) {
        const int64_t block = (kWhole ? i : min(i, n - 1)) / kAdamwBlock;
        decode_e4m3(load_codes(t.m, i, n, wide), t.m_scale[block], m);
        decode_e4m3(load_codes(t.v, i, n, wide), t.v_scale[block], v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= v[k];
    } else {
        load8<true>(t.m, i, n, wide, m);
        load8<true>(t.v, i, n, wide, v);
    }
    // The moments in single roundings, in the order the formula has them: an 8-bit code jumps by a
    // sixteenth where its value crosses a midpoint, so a value that another evaluation in fp32
    // reproduces is worth more than the fused product that is nearer.  The parameter has no such
    // borders.
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float gk = __fmul_rn(g[k], h.grad_scale);
        m[k] = __fadd_rn(__fmul_rn(h.beta1, m[k]), __fmul_rn(h.one_beta1, gk));
        v[k] = __fadd_rn(__fmul_rn(h.beta2, v[k]), __fmul_rn(__fmul_rn(h.one_beta2, gk), gk));
    }
    if (kState8) {
        sqrt8(v, r);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = __fsqrt_rn(v[k]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(fmaf(r[k], h.inv_root_c2, h.eps)));
        p[k] -= h.step_c1 * m[k] * inv + h.decay * p[k];
    }
    if (t.master != nullptr) store8<true>(t.master, i, n, wide, p);
    store8<kPF32>(t.p, i, n, wide, p);
    if (kState8) {
        float ms, vs;
        // 8 x 16 bits for each moment: counter (i / 8, tensor, step, i / 2^35 and the moment in the top bit)
        uint4 mb = make_uint4(0u, 0u, 0u, 0u), vb = mb;
        if (kSr) {
            const uint32_t lo = static_cast<uint32_t>(i >> 3), hi = static_cast<uint32_t>(i >> 35);
            mb = philox4x32_10(lo, h.tensor, h.step, hi, h.seed);
            vb = philox4x32_10(lo, h.tensor, h.step, hi | 0x80000000u, h.seed);
        }
        const uint2 mq = encode_block<false, kSr>(m, &ms, mb), vq = encode_block<true, kSr>(r, &vs, vb);
        store_codes(t.m, i, n, wide, mq);
        store_codes(t.v, i, n, wide, vq);
        if ((threadIdx.x & 15) == 0 && (kWhole || i < n)) {
            t.m_scale[i / kAdamwBlock] = ms;
            t.v_scale[i / kAdamwBlock] = vs;
        }
    } else {
        store8<true>(t.m, i, n, wide, m);
        store8<true>(t.v, i, n, wide, v);
    }
}

template <bool kPF32, bool kGF32, bool kState8, bool kSr, int kCap>
__global__ void __launch_bounds__(kState8 ? kThreads8 : kThreads32, kState8 ? 32 : 8) adamw_kernel(const __grid_constant__ AdamwArgs<kCap> a) {
    grid_wait_prerequisites();
    grid_launch_dependents();
    const int unit = static_cast<int>(blockIdx.x);
    int lo = 0, hi = a.count - 1;   // the tensor of this unit: the first with end > unit
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.end[mid] > unit) hi = mid;
        else lo = mid + 1;
    }
    const mxfp4_adamw_tensor& t = a.t[lo];
    const int64_t n = t.n;
    const int64_t base = static_cast<int64_t>(unit - (lo > 0 ? a.end[lo - 1] : 0)) * kAdamwUnit;
    const bool dyn = a.dynamic != nullptr;
    const float lr = dyn ? __ldg(a.dynamic) : a.lr;
    const float c1 = dyn ? __ldg(a.dynamic + 1) : a.c1, c2 = dyn ? __ldg(a.dynamic + 2) : a.c2;
    Hyper h{a.beta1, a.one_beta1, a.beta2, a.one_beta2, a.eps, lr / c1, 1.0f / sqrtf(c2), lr * a.weight_decay,
            dyn ? __ldg(a.dynamic + 3) : a.grad_scale, 0u, 0u, 0u};
    if (kSr) {
        h.tensor = static_cast<uint32_t>(a.first + lo);
        h.step = dyn ? static_cast<uint32_t>(__ldg(a.dynamic + 4)) : a.step;
        h.seed = a.seed;
    }
    // every pointer where an 8-element access may start: 16 bytes apart (codes: 8)
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.p) | reinterpret_cast<uintptr_t>(t.g) |
                          reinterpret_cast<uintptr_t>(t.master) |
                          (kState8 ? (reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v)) << 1
                                   : reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v));
    const bool aligned = (all & 15u) == 0;
    const int64_t i0 = base + 8 * threadIdx.x;
    constexpr int kPass = 8 * (kState8 ? kThreads8 : kThreads32);
    if (aligned && base + kAdamwUnit <= n) {
#pragma unroll 1
        for (int k = 0; k < kAdamwUnit; k += kPass) update8<kPF32, kGF32, kState8, kSr, true>(t, h, i0 + k, n, true);
    } else {
#pragma unroll 1
        for (int k = 0; k < kAdamwUnit; k += kPass) update8<kPF32, kGF32, kState8, kSr, false>(t, h, i0 + k, n, aligned);
    }
}

template <int kCap>
cudaError_t launch(const AdamwArgs<kCap>& a, int flags, cudaStream_t stream) {
    using K = void (*)(AdamwArgs<kCap>);
    static const K kernels[16] = {
        adamw_kernel<false, false, false, false, kCap>, adamw_kernel<true, false, false, false, kCap>,
        adamw_kernel<false, true, false, false, kCap>,  adamw_kernel<true, true, false, false, kCap>,
        adamw_kernel<false, false, true, false, kCap>,  adamw_kernel<true, false, true, false, kCap>,
        adamw_kernel<false, true, true, false, kCap>,   adamw_kernel<true, true, true, false, kCap>,
        nullptr, nullptr, nullptr, nullptr,   // stochastic rounding is of 8-bit moments
        adamw_kernel<false, false, true, true, kCap>,   adamw_kernel<true, false, true, true, kCap>,
        adamw_kernel<false, true, true, true, kCap>,    adamw_kernel<true, true, true, true, kCap>};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.end[a.count - 1]), 1, 1);
    cfg.blockDim = dim3(flags & MXFP4_ADAMW_STATE_E4M3 ? kThreads8 : kThreads32, 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernels[flags], a);
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

mxfp4_status check(int32_t count, const mxfp4_adamw_tensor* t, int32_t flags, const mxfp4_adamw_params* h) {
    if (count < 0 || (count > 0 && t == nullptr) || h == nullptr || (flags & ~15)) return MXFP4_ERR_INVALID_ARG;
    if ((flags & MXFP4_ADAMW_STOCHASTIC) && !(flags & MXFP4_ADAMW_STATE_E4M3)) return MXFP4_ERR_INVALID_ARG;
    // the fp32 values that the kernel uses have to lie in the ranges too
    const float b1 = static_cast<float>(h->beta1), b2 = static_cast<float>(h->beta2), eps = static_cast<float>(h->eps);
    if (!(h->beta1 >= 0.0 && b1 < 1.0f) || !(h->beta2 >= 0.0 && b2 < 1.0f) || !(h->eps >= 0.0) || h->step < 1 ||
        !std::isfinite(eps) || (h->eps > 0.0 && eps < kMinScale) || !std::isfinite(h->lr) || !std::isfinite(h->weight_decay))
        return MXFP4_ERR_INVALID_ARG;
    if (!aligned_to(h->dynamic, 4)) return MXFP4_ERR_MISALIGNED;
    const bool p_f32 = flags & MXFP4_ADAMW_P_F32, g_f32 = flags & MXFP4_ADAMW_G_F32, s8 = flags & MXFP4_ADAMW_STATE_E4M3;
    for (int32_t j = 0; j < count; ++j) {
        const mxfp4_adamw_tensor& x = t[j];
        if (x.n < 0 || x.n > (int64_t{1} << 40)) return MXFP4_ERR_INVALID_ARG;
        if (p_f32 && x.master != nullptr) return MXFP4_ERR_INVALID_ARG;
        if (x.n > 0 && (!x.p || !x.g || !x.m || !x.v || (s8 && (!x.m_scale || !x.v_scale)))) return MXFP4_ERR_INVALID_ARG;
        if (!aligned_to(x.p, p_f32 ? 4 : 2) || !aligned_to(x.g, g_f32 ? 4 : 2) || !aligned_to(x.master, 4) ||
            !aligned_to(x.m, s8 ? 1 : 4) || !aligned_to(x.v, s8 ? 1 : 4) ||
            (s8 && (!aligned_to(x.m_scale, 4) || !aligned_to(x.v_scale, 4))))
            return MXFP4_ERR_MISALIGNED;
    }
    // codes rounded to nearest do not follow a slower second moment (the head of this file)
    if (s8 && !(flags & MXFP4_ADAMW_STOCHASTIC) && h->beta2 > kNearestBeta2) return MXFP4_ERR_INVALID_ARG;
    return MXFP4_OK;
}

template <int kCap>
mxfp4_status step(int32_t count, const mxfp4_adamw_tensor* t, int32_t flags, const mxfp4_adamw_params& h,
                  cudaStream_t stream) {
    AdamwArgs<kCap> a;
    a.beta1 = static_cast<float>(h.beta1);
    a.one_beta1 = static_cast<float>(1.0 - h.beta1);
    a.beta2 = static_cast<float>(h.beta2);
    a.one_beta2 = static_cast<float>(1.0 - h.beta2);
    a.eps = static_cast<float>(h.eps);
    a.weight_decay = static_cast<float>(h.weight_decay);
    a.lr = static_cast<float>(h.lr);
    a.c1 = static_cast<float>(1.0 - std::pow(h.beta1, static_cast<double>(h.step)));
    a.c2 = static_cast<float>(1.0 - std::pow(h.beta2, static_cast<double>(h.step)));
    a.grad_scale = static_cast<float>(h.grad_scale);
    a.dynamic = h.dynamic;
    a.first = 0;
    a.step = static_cast<uint32_t>(h.step);
    a.seed = flags & MXFP4_ADAMW_STOCHASTIC ? h.seed : 0;
    int32_t j = 0;
    while (j < count) {
        int64_t units = 0;
        a.count = 0;
        while (j < count && a.count < kCap) {
            if (t[j].n == 0) {
                ++j;
                continue;
            }
            const int64_t more = (t[j].n + kAdamwUnit - 1) / kAdamwUnit;
            if (units + more > 0x7FFFFFFF) break;
            units += more;
            a.t[a.count] = t[j++];
            a.end[a.count++] = static_cast<int32_t>(units);
        }
        if (a.count > 0 && launch<kCap>(a, flags, stream) != cudaSuccess) return MXFP4_ERR_CUDA;
        a.first += a.count;
    }
    return MXFP4_OK;
}

}  // namespace
}  // namespace mxfp4

extern "C" mxfp4_status mxfp4_adamw(int32_t count, const mxfp4_adamw_tensor* tensors, int32_t flags,
                                    const mxfp4_adamw_params* params, mxfp4_stream_t stream) {
    const mxfp4_status ok = mxfp4::check(count, tensors, flags, params);
    if (ok != MXFP4_OK) return ok;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK) return static_cast<mxfp4_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return count <= mxfp4::kAdamwFew ? mxfp4::step<mxfp4::kAdamwFew>(count, tensors, flags, *params, s)
                                     : mxfp4::step<mxfp4::kAdamwMany>(count, tensors, flags, *params, s);
}
