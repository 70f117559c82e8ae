// grad_norm.cu -- the norm of all gradients of a step, and scaling them by a factor on the device.
//
//   norm = sqrt(sum over all tensors of sum g^2),  factor = min(1, max_norm / (norm + 1e-6)),
//   and, for clipping in place, g = factor g, in fp32 and rounded to its type.
//
// Sums.  A thread adds the squares of 32 elements (fp32: 16) in fp32 and everything above that in fp64: the
// norm is off by a few 2^-24 at most however many elements there are, and the order is fixed, so
// the same gradients give the same bits.  Squares leave fp32's range where the elements do not
// (1e20, or 1e-25 throughout): a sum of 32 above 2^120 or below 2^-80 is formed again from the
// registers with the elements times 2^-80 or 2^80, both exact up to what cannot count.
//
// The norm is bound by the memory: 2 or 4 bytes an element, and about 1.5 instructions (bf16: 140 M elements in
// 47 us, 6.0 TB/s; 288 M in 88 us, 6.5 TB/s).  Clipping in place reads and writes the gradients once more, and runs
// through them backward, so that what the norm read last is still in the L2 (129 MB): 288 M in 272 us, 1.73 GB of traffic
// at 6.4 TB/s.  (Loads and stores that ask not to be kept there, so that more of it stays, made both passes slower.)
//
// Work.  A unit of 16 KB, at addresses that are multiples of 16 bytes whatever the tensor's own
// alignment: a tensor's first unit leaves out what lies before it.  A CTA takes a range of consecutive
// units, each one's loads under way while the one before is added up.  The last CTA to leave its sum
// adds them all up; nobody waits for anybody.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "launch.h"
#include "launch_grad_norm.h"
#include "ptx.cuh"

namespace mxfp4 {
namespace {

constexpr float kBig = 1.329227996e36f;        // 2^120
constexpr float kSmall = 8.271806126e-25f;     // 2^-80
constexpr float kUp = 1.208925820e24f;         // 2^80
constexpr double kUp2 = 1.461501637330902918e48;       // 2^160
constexpr double kSmall2 = 6.842277657836020854e-49;   // 2^-160
constexpr int kLoads = kGradUnitBytes / kGradThreads / 16;   // 16-byte loads of a thread's part

template <bool kF32>
constexpr int kElements = kGradUnitBytes / (kF32 ? 4 : 2);   // of a unit

// A walk through consecutive units, in either direction: the tensor of each and the element at which it starts
// (below zero, by less than a load, in a tensor's first unit).
template <bool kF32, int kCap>
struct Walk {
    const GradArgs<kCap>& a;
    int j;          // tensor
    void* g;
    int64_t n, first;

    __device__ __forceinline__ Walk(const GradArgs<kCap>& args, int unit) : a(args) {
        int lo = 0, hi = a.count - 1;   // the first tensor with end > unit
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.end[mid] > unit) hi = mid;
            else lo = mid + 1;
        }
        j = lo;
        at(unit);
    }
    __device__ __forceinline__ void at(int unit) {
        g = a.t[j].g;
        n = a.t[j].n;
        const int skew = static_cast<int>(reinterpret_cast<uintptr_t>(g) & 15u) / (kF32 ? 4 : 2);
        first = static_cast<int64_t>(unit - (j > 0 ? a.end[j - 1] : 0)) * kElements<kF32> - skew;
    }
    __device__ __forceinline__ void up(int unit) {
        if (unit >= a.end[j]) {
            ++j;
            at(unit);
        } else {
            first += kElements<kF32>;
        }
    }
    __device__ __forceinline__ void down(int unit) {
        if (j > 0 && unit < a.end[j - 1]) {
            --j;
            at(unit);
        } else {
            first -= kElements<kF32>;
        }
    }
};

// A thread's part of the unit at `first`, as 32-bit words: pairs of bf16, or fp32.
template <bool kF32>
struct Part {
    static constexpr int kPer = kF32 ? 4 : 8;     // elements of a load
    static constexpr int kElement = kF32 ? 4 : 2;
    uint4 w[kLoads];

    __device__ __forceinline__ static int64_t at(int64_t first, int j) {
        return first + (j * kGradThreads + static_cast<int>(threadIdx.x)) * kPer;
    }
    __device__ __forceinline__ static uint32_t load1(const void* g, int64_t i) {
        return kF32 ? static_cast<const uint32_t*>(g)[i] : static_cast<const uint16_t*>(g)[i];
    }
    __device__ __forceinline__ void load(const void* g, int64_t n, int64_t first) {
        if (first >= 0 && first + kElements<kF32> <= n) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                w[j] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g) + at(first, j) * kElement);
            return;
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t i = at(first, j);
            w[j] = make_uint4(0u, 0u, 0u, 0u);
            if (i >= 0 && i + kPer <= n) {
                w[j] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(g) + i * kElement);
            } else if (i + kPer > 0 && i < n) {
                uint32_t* const v = reinterpret_cast<uint32_t*>(&w[j]);
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (i + k >= 0 && i + k < n) {
                        if (kF32) v[k] = load1(g, i + k);
                        else v[k >> 1] |= load1(g, i + k) << (16 * (k & 1));
                    }
            }
        }
    }
    __device__ __forceinline__ float sum(float scale) const {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const uint32_t v[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kF32) {
                    const float a = __uint_as_float(v[k]) * scale;
                    s[k] = fmaf(a, a, s[k]);
                } else {
                    const float a = __uint_as_float(v[k] << 16) * scale, b = __uint_as_float(v[k] & 0xFFFF0000u) * scale;
                    s[k] = fmaf(a, a, s[k]);
                    s[k] = fmaf(b, b, s[k]);
                }
            }
        }
        return (s[0] + s[1]) + (s[2] + s[3]);
    }
    __device__ __forceinline__ bool any() const {
        uint32_t o = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) o |= w[j].x | w[j].y | w[j].z | w[j].w;
        return (o & (kF32 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) != 0;
    }
    __device__ __forceinline__ double squares() const {
        const float s = sum(1.0f);
        if (s >= kSmall && s <= kBig) return static_cast<double>(s);
        if (s < kSmall) return any() ? static_cast<double>(sum(kUp)) * kSmall2 : 0.0;
        return static_cast<double>(sum(kSmall)) * kUp2;   // NaN and infinities too
    }
    __device__ __forceinline__ void scale(float f) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            uint32_t* const v = reinterpret_cast<uint32_t*>(&w[j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (kF32) {
                    v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(v[k] << 16) * f,
                                                                   __uint_as_float(v[k] & 0xFFFF0000u) * f);
                    v[k] = *reinterpret_cast<const uint32_t*>(&h);
                }
            }
        }
    }
    __device__ __forceinline__ void store(void* g, int64_t n, int64_t first) const {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t i = at(first, j);
            if (i >= 0 && i + kPer <= n) {
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(g) + i * kElement) = w[j];
            } else if (i + kPer > 0 && i < n) {
                const uint32_t* const v = reinterpret_cast<const uint32_t*>(&w[j]);
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (i + k >= 0 && i + k < n) {
                        if (kF32) static_cast<uint32_t*>(g)[i + k] = v[k];
                        else static_cast<uint16_t*>(g)[i + k] = static_cast<uint16_t>(v[k >> 1] >> (16 * (k & 1)));
                    }
            }
        }
    }
};

// The first of the units of CTA `cta`.
__device__ __forceinline__ int range_start(int units, int cta) {
    return static_cast<int>(static_cast<int64_t>(units) * cta / gridDim.x);
}

// The CTA's sum of x, in thread 0; every thread calls it.
__device__ __forceinline__ double block_sum(double x, double* shared) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    __syncthreads();
    if (lane_id() == 0) shared[threadIdx.x >> 5] = x;
    __syncthreads();
    if (threadIdx.x < 32) {
        x = lane_id() < kGradThreads / 32 ? shared[lane_id()] : 0.0;
#pragma unroll
        for (int d = kGradThreads / 64; d > 0; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
    }
    return x;
}

template <bool kF32, int kCap>
__global__ void __launch_bounds__(kGradThreads, kGradCtasPerSm) grad_norm_kernel(const __grid_constant__ GradArgs<kCap> a) {
    __shared__ double shared[kGradThreads / 32];
    __shared__ bool last;
    grid_wait_prerequisites();
    grid_launch_dependents();
    const int units = a.end[a.count - 1];
    int u = range_start(units, blockIdx.x);
    const int end = range_start(units, blockIdx.x + 1);   // above u: there are no more CTAs than units
    double sum = 0.0;
    Walk<kF32, kCap> w(a, u);
    Part<kF32> next;
    next.load(w.g, w.n, w.first);
    for (; u < end; ++u) {
        const Part<kF32> p = next;
        if (u + 1 < end) {
            w.up(u + 1);
            next.load(w.g, w.n, w.first);
        }
        sum += p.squares();
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) {
        a.partial[a.slot + blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(&a.head->done, 1u) == static_cast<uint32_t>(a.slots) - 1u;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    sum = 0.0;
    for (int i = threadIdx.x; i < a.slots; i += kGradThreads) sum += __ldcg(a.partial + i);
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        double factor = a.max_norm / (norm + 1e-6);
        if (factor > 1.0 || isinf(a.max_norm)) factor = 1.0;
        if (isnan(norm)) factor = norm;   // whatever max_norm is
        a.out[0] = static_cast<float>(norm);
        a.out[1] = static_cast<float>(factor);
        a.head->done = 0;
    }
}

template <bool kF32, int kCap>
__global__ void __launch_bounds__(kGradThreads, kGradCtasPerSm) grad_scale_kernel(const __grid_constant__ GradArgs<kCap> a) {
    grid_wait_prerequisites();
    grid_launch_dependents();
    const float factor = __ldcg(a.out + 1);
    const int units = a.end[a.count - 1];
    const int start = range_start(units, blockIdx.x);
    int u = range_start(units, blockIdx.x + 1) - 1;
    Walk<kF32, kCap> w(a, u);
    Part<kF32> next;
    next.load(w.g, w.n, w.first);
    for (; u >= start; --u) {
        Part<kF32> p = next;
        void* const g = w.g;
        const int64_t n = w.n, first = w.first;
        if (u > start) {
            w.down(u - 1);
            next.load(w.g, w.n, w.first);
        }
        p.scale(factor);
        p.store(g, n, first);
    }
}

__global__ void grad_empty_kernel(float* out) {
    grid_wait_prerequisites();
    grid_launch_dependents();
    out[0] = 0.0f;
    out[1] = 1.0f;
}

template <typename Kernel, typename Args>
cudaError_t launch(Kernel kernel, const Args& a, int ctas, int threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

inline int64_t units_of(const mxfp4_grad_tensor& t, int esize) {
    const int64_t skew = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.g) & 15u) / esize;
    const int64_t unit = kGradUnitBytes / esize;
    return (t.n + skew + unit - 1) / unit;
}

// The tensors from t[j] on that one launch takes, and the index behind them and the empty ones that follow; none are left: count 0.
template <int kCap>
int32_t fill(GradArgs<kCap>* a, int32_t count, const mxfp4_grad_tensor* t, int32_t j, int esize) {
    int64_t units = 0;   // below 2^29: check() bounds the elements of a call
    a->count = 0;
    for (; j < count; ++j) {
        if (t[j].n == 0) continue;
        if (a->count == kCap) break;
        units += units_of(t[j], esize);
        a->t[a->count] = t[j];
        a->end[a->count++] = static_cast<int32_t>(units);
    }
    return j;
}

inline int ctas_of(int units, int sms) {
    const int most = kGradCtasPerSm * (sms < kGradMaxSms ? sms : kGradMaxSms);
    return units < most ? units : most;
}

template <bool kF32, int kCap>
mxfp4_status run(int32_t count, const mxfp4_grad_tensor* t, double max_norm, float* out, void* workspace, bool scale,
                 int sms, cudaStream_t stream) {
    GradArgs<kCap> a;
    const int esize = kF32 ? 4 : 2;
    a.head = static_cast<GradHead*>(workspace);
    a.partial = reinterpret_cast<double*>(a.head + 1);
    a.max_norm = max_norm;
    a.out = out;
    a.slots = 0;
    int32_t starts[kGradLaunches], launches = 0;
    for (int32_t j = 0; j < count;) {
        starts[launches] = j;
        j = fill(&a, count, t, j, esize);
        if (a.count == 0) break;
        a.slots += ctas_of(a.end[a.count - 1], sms);
        ++launches;
    }
    if (launches == 0) return launch(grad_empty_kernel, out, 1, 1, stream) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
    a.slot = 0;
    for (int32_t i = 0; i < launches; ++i) {
        if (launches > 1) fill(&a, count, t, starts[i], esize);
        const int ctas = ctas_of(a.end[a.count - 1], sms);
        if (launch(grad_norm_kernel<kF32, kCap>, a, ctas, kGradThreads, stream) != cudaSuccess) return MXFP4_ERR_CUDA;
        a.slot += ctas;
    }
    if (!scale) return MXFP4_OK;
    for (int32_t i = launches - 1; i >= 0; --i) {   // what was read last first
        if (launches > 1) fill(&a, count, t, starts[i], esize);
        if (launch(grad_scale_kernel<kF32, kCap>, a, ctas_of(a.end[a.count - 1], sms), kGradThreads, stream) != cudaSuccess)
            return MXFP4_ERR_CUDA;
    }
    return MXFP4_OK;
}

// No two of the tensors share an element.  Most lists are in the order of their addresses already, or in the opposite one.
mxfp4_status check_apart(int32_t count, const mxfp4_grad_tensor* t, uintptr_t esize) {
    const auto from = [&](const mxfp4_grad_tensor& x) { return reinterpret_cast<uintptr_t>(x.g); };
    const auto to = [&](const mxfp4_grad_tensor& x) { return from(x) + static_cast<uintptr_t>(x.n) * esize; };
    bool up = true, down = true;
    const mxfp4_grad_tensor* before = nullptr;
    for (int32_t j = 0; j < count && (up || down); ++j) {
        if (t[j].n == 0) continue;
        if (before != nullptr) {
            up = up && to(*before) <= from(t[j]);
            down = down && to(t[j]) <= from(*before);
        }
        before = &t[j];
    }
    if (up || down) return MXFP4_OK;
    int32_t* const order = new (std::nothrow) int32_t[count];
    if (order == nullptr) return MXFP4_ERR_CUDA;
    int32_t n = 0;
    for (int32_t j = 0; j < count; ++j)
        if (t[j].n > 0) order[n++] = j;
    std::sort(order, order + n, [&](int32_t a, int32_t b) { return from(t[a]) < from(t[b]); });
    bool apart = true;
    for (int32_t j = 1; j < n; ++j) apart = apart && to(t[order[j - 1]]) <= from(t[order[j]]);
    delete[] order;
    return apart ? MXFP4_OK : MXFP4_ERR_INVALID_ARG;
}

mxfp4_status check(int32_t count, const mxfp4_grad_tensor* t, int32_t flags, double max_norm, const float* out,
                   const void* workspace, size_t bytes) {
    size_t need = 0;
    if (mxfp4_grad_norm_workspace_bytes(count, &need) != MXFP4_OK || (count > 0 && t == nullptr) || (flags & ~3) ||
        !(max_norm > 0.0) || out == nullptr || workspace == nullptr || bytes < need)
        return MXFP4_ERR_INVALID_ARG;
    const uintptr_t element = flags & MXFP4_GRAD_F32 ? 4 : 2;
    int64_t total = 0;
    for (int32_t j = 0; j < count; ++j) {
        if (t[j].n < 0 || t[j].n > (int64_t{1} << 40) || (t[j].n > 0 && t[j].g == nullptr)) return MXFP4_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(t[j].g) & (element - 1)) return MXFP4_ERR_MISALIGNED;
        total += t[j].n;
        if (total > int64_t{1} << 40) return MXFP4_ERR_INVALID_ARG;
    }
    if (flags & MXFP4_GRAD_SCALE) {
        const mxfp4_status apart = check_apart(count, t, element);
        if (apart != MXFP4_OK) return apart;
    }
    if ((reinterpret_cast<uintptr_t>(out) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MXFP4_ERR_MISALIGNED;
    return MXFP4_OK;
}

}  // namespace
}  // namespace mxfp4

extern "C" {

mxfp4_status mxfp4_grad_norm_workspace_bytes(int32_t count, size_t* bytes) {
    if (count < 0 || count > MXFP4_GRAD_MAX_TENSORS || bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
    const size_t launches = static_cast<size_t>(count) / mxfp4::kGradMany + 1;
    *bytes = sizeof(mxfp4::GradHead) + launches * mxfp4::kGradSlots * sizeof(double);
    return MXFP4_OK;
}

mxfp4_status mxfp4_grad_norm(int32_t count, const mxfp4_grad_tensor* tensors, int32_t flags, double max_norm, float* out,
                             void* workspace, size_t workspace_bytes, mxfp4_stream_t stream) {
    const mxfp4_status ok = mxfp4::check(count, tensors, flags, max_norm, out, workspace, workspace_bytes);
    if (ok != MXFP4_OK) return ok;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK) return static_cast<mxfp4_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool scale = flags & MXFP4_GRAD_SCALE, f32 = flags & MXFP4_GRAD_F32, few = count <= mxfp4::kGradFew;
    if (f32)
        return few ? mxfp4::run<true, mxfp4::kGradFew>(count, tensors, max_norm, out, workspace, scale, sms, s)
                   : mxfp4::run<true, mxfp4::kGradMany>(count, tensors, max_norm, out, workspace, scale, sms, s);
    return few ? mxfp4::run<false, mxfp4::kGradFew>(count, tensors, max_norm, out, workspace, scale, sms, s)
               : mxfp4::run<false, mxfp4::kGradMany>(count, tensors, max_norm, out, workspace, scale, sms, s);
}

}  // extern "C"
