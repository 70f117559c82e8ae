// norm_forward.cu -- layer norm of the rows of X.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r g + b, g = w or 1 + w,
//   with w and b for the whole of X, for each sample of it (consecutive rows), or not at all.
//
// A row is read once and stays in registers: the sum, then the sum of the squares of the centred
// values.  The sum of the centred values themselves goes with them and corrects the mean by what its
// own rounding and the first sum's left, which counts where |mu| is far above the deviation.  All
// of it in fp32; y is rounded once.  Bound by the memory.
//
// A warp takes a row of up to 1024 elements, a CTA a longer one, 16 elements a thread.  CTAs stay for
// many rows, with the vectors in registers, and load their next row before they work on this one.
#include <atomic>

#include "norm_row.cuh"

namespace mxfp4 {
namespace {

template <bool kF32, bool kWide, int kGroups, bool kWarpRow, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float2 shared[2][32];
    using Part = RowPart<kF32, kWide, kGroups>;
    constexpr int kE = Part::kElements;
    constexpr int kSize = kF32 ? 4 : 2;
    const int t = kWarpRow ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const int threads = kWarpRow ? 32 : static_cast<int>(blockDim.x);
    const int64_t stride = kWarpRow ? static_cast<int64_t>(gridDim.x) * (kThreads / 32) : gridDim.x;
    int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const float inv = 1.0f / static_cast<float>(a.dim);
    grid_wait_prerequisites();
    grid_launch_dependents();
    float g[kE], b[kE];
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        g[k] = 1.0f;
        b[k] = 0.0f;
    }
    int64_t sample = -1;
    Part next;
    if (row < a.rows) next.load(static_cast<const uint8_t*>(a.x) + row * a.ldx * kSize, a.dim, t, threads);
    for (; row < a.rows; row += stride) {
        const Part x = next;
        if (row + stride < a.rows) next.load(static_cast<const uint8_t*>(a.x) + (row + stride) * a.ldx * kSize, a.dim, t, threads);
        const int64_t s = row < a.sample_rows ? 0 : row / a.sample_rows;
        if (s != sample) {
            sample = s;
            if (a.weight != nullptr) {
                load_vector<kWide, kGroups>(a.weight, s * a.dim, a.w_f32, a.dim, t, threads, g);
                if (a.add_one)
#pragma unroll
                    for (int k = 0; k < kE; ++k) g[k] += 1.0f;
            }
            if (a.bias != nullptr) load_vector<kWide, kGroups>(a.bias, s * a.dim, a.w_f32, a.dim, t, threads, b);
        }
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kE; ++k) sum.x += x.get(k);
        sum = row_sum2<kWarpRow>(sum, shared[0]);
        float mean = sum.x * inv;
        sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kE; ++k) {
            const float d = Part::column(k, t, threads) < a.dim ? x.get(k) - mean : 0.0f;
            sum.x += d;
            sum.y = fmaf(d, d, sum.y);
        }
        sum = row_sum2<kWarpRow>(sum, shared[1]);
        const float rest = sum.x * inv;
        mean += rest;
        const float rstd = 1.0f / sqrtf(fmaxf(fmaf(-rest, rest, sum.y * inv), 0.0f) + a.eps);
        float y[kE];
#pragma unroll
        for (int k = 0; k < kE; ++k) y[k] = fmaf((x.get(k) - mean) * rstd, g[k], b[k]);
        Part::store(static_cast<uint8_t*>(a.y) + row * a.ldy * kSize, y, a.dim, t, threads);
        if (a.mean != nullptr && t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

bool wide(const NormArgs& a) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                          reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.bias);
    return (all & 15u) == 0 && a.dim % 8 == 0 && (a.rows == 1 || (a.ldx % 8 == 0 && a.ldy % 8 == 0));
}

template <bool kF32, bool kWide, int kGroups, bool kWarpRow, int kThreads>
cudaError_t launch(const NormArgs& a, int sms, cudaStream_t stream) {
    const auto kernel = norm_forward_kernel<kF32, kWide, kGroups, kWarpRow, kThreads>;
    const int threads = kWarpRow ? kThreads : ((a.dim + 8 * kGroups - 1) / (8 * kGroups) + 31) / 32 * 32;
    const int64_t need = kWarpRow ? (a.rows + kThreads / 32 - 1) / (kThreads / 32) : a.rows;
    static std::atomic<int> per_sm[kThreads / 32 + 1];   // resident CTAs an SM, by warps of the CTA
    int n = per_sm[threads / 32].load(std::memory_order_relaxed);
    if (n == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        per_sm[threads / 32].store(n, std::memory_order_relaxed);
    }
    const int64_t most = static_cast<int64_t>(n) * sms;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(need < most ? need : most), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kF32, bool kWide>
cudaError_t launch(const NormArgs& a, int sms, cudaStream_t stream) {
    if (a.dim <= 256) return launch<kF32, kWide, 1, true, 256>(a, sms, stream);
    if (a.dim <= 512) return launch<kF32, kWide, 2, true, 256>(a, sms, stream);
    if (a.dim <= kNormWarpRowDim) return launch<kF32, kWide, 4, true, 256>(a, sms, stream);
    if (a.dim <= 4096) return launch<kF32, kWide, 2, false, 256>(a, sms, stream);
    if (a.dim <= 8192) return launch<kF32, kWide, 2, false, 512>(a, sms, stream);
    return launch<kF32, kWide, 2, false, 1024>(a, sms, stream);
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, bool f32, int sms, cudaStream_t stream) {
    if (wide(a)) return f32 ? launch<true, true>(a, sms, stream) : launch<false, true>(a, sms, stream);
    return f32 ? launch<true, false>(a, sms, stream) : launch<false, false>(a, sms, stream);
}

}  // namespace mxfp4
