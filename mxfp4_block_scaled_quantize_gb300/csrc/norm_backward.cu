// norm_backward.cu -- the backward pass of layer norm, with the gradients of its weight and bias.
//
// With xh = (x - mu) r and a = dy g (g = w or 1 + w):
//   dx = r (a - mean(a) - xh mean(a xh)),  dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// One pass over X and dY: a CTA takes a range of consecutive rows of one sample (rows of up to 1024
// elements: a warp each), keeps its columns' sums of dw and db in registers across them, and
// leaves them as one partial row; a second kernel adds the partial rows in a fixed order, so the same
// inputs give the same bits.  A sample that is one CTA's needs no second kernel.  Bound by the
// memory: x and dy in, dx out; the partial rows are 2 / chunk_rows of that.
#include "norm_row.cuh"

namespace mxfp4 {
namespace {

template <bool kF32, bool kWide, int kGroups, bool kWarpRow, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(const __grid_constant__ NormArgs a) {
    using Part = RowPart<kF32, kWide, kGroups>;
    constexpr int kE = Part::kElements;
    constexpr int kSize = kF32 ? 4 : 2;
    constexpr int kWarps = kThreads / 32;
    __shared__ float2 shared[2][32];
    __shared__ float sums[kWarpRow ? kWarps : 1][kWarpRow ? 32 * kE : 1];
    const int t = kWarpRow ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const int threads = kWarpRow ? 32 : static_cast<int>(blockDim.x);
    const int64_t sample = blockIdx.x / a.chunks;
    const int64_t in_sample = static_cast<int64_t>(blockIdx.x % a.chunks) * a.chunk_rows;
    const int64_t first = sample * a.sample_rows + in_sample;
    const int64_t end = sample * a.sample_rows + min(in_sample + a.chunk_rows, a.sample_rows);
    const int64_t stride = kWarpRow ? kWarps : 1;
    const float inv = 1.0f / static_cast<float>(a.dim);
    grid_wait_prerequisites();
    grid_launch_dependents();
    float g[kE], dw[kE], db[kE];
#pragma unroll
    for (int k = 0; k < kE; ++k) {
        g[k] = 1.0f;
        dw[k] = 0.0f;
        db[k] = 0.0f;
    }
    if (a.weight != nullptr) {
        load_vector<kWide, kGroups>(a.weight, sample * a.dim, a.w_f32, a.dim, t, threads, g);
        if (a.add_one)
#pragma unroll
            for (int k = 0; k < kE; ++k) g[k] += 1.0f;
    }
    int64_t row = first + (kWarpRow ? threadIdx.x >> 5 : 0);
    Part nx, ny;
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t r) {
        nx.load(static_cast<const uint8_t*>(a.x) + r * a.ldx * kSize, a.dim, t, threads);
        ny.load(static_cast<const uint8_t*>(a.dy) + r * a.lddy * kSize, a.dim, t, threads);
        nmean = __ldg(a.mean + r);
        nrstd = __ldg(a.rstd + r);
    };
    if (row < end) fetch(row);
    int turn = 0;
    for (; row < end; row += stride, turn ^= 1) {
        const Part x = nx, y = ny;
        const float mean = nmean, rstd = nrstd;
        if (row + stride < end) fetch(row + stride);
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kE; ++k) {   // dy is zero behind the row's end
            const float xh = (x.get(k) - mean) * rstd, d = y.get(k), c = d * g[k];
            dw[k] = fmaf(d, xh, dw[k]);
            db[k] += d;
            sum.x += c;
            sum.y = fmaf(c, xh, sum.y);
        }
        sum = row_sum2<kWarpRow>(sum, shared[turn]);
        const float m1 = sum.x * inv, m2 = sum.y * inv;
        float out[kE];
#pragma unroll
        for (int k = 0; k < kE; ++k) {
            const float xh = (x.get(k) - mean) * rstd;
            out[k] = rstd * (fmaf(-xh, m2, y.get(k) * g[k]) - m1);
        }
        Part::store(static_cast<uint8_t*>(a.y) + row * a.ldy * kSize, out, a.dim, t, threads);
    }
    float* const to[2] = {a.partial_w, a.partial_b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (to[i] == nullptr) continue;
        float* const out = to[i] + static_cast<int64_t>(blockIdx.x) * a.dim;
        const float* const v = i == 0 ? dw : db;
        if (kWarpRow) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kE; ++k) sums[threadIdx.x >> 5][kWide ? Part::column(k, t, 32) : k * 32 + t] = v[k];
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sums[w][c];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kE; ++k) {
                const int c = Part::column(k, t, threads);
                if (c < a.dim) out[c] = v[k];
            }
        }
    }
}

// Sums of the partial rows: 32 columns of one sample a CTA, 8 strips of its partial rows.
constexpr int kStrips = 8;
__global__ void __launch_bounds__(32 * kStrips) norm_reduce_kernel(const __grid_constant__ NormReduceArgs a) {
    __shared__ float sums[kStrips][33];
    grid_wait_prerequisites();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, strip = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    for (int64_t s = blockIdx.y; s < a.samples; s += gridDim.y) {
        const float* const p = a.partial[blockIdx.z] + s * a.chunks * a.dim;
        float v = 0.0f;
        if (c < a.dim)
#pragma unroll 8
            for (int i = strip; i < a.chunks; i += kStrips) v += __ldcg(p + static_cast<int64_t>(i) * a.dim + c);
        __syncthreads();
        sums[strip][lane] = v;
        __syncthreads();
        if (strip == 0 && c < a.dim) {
#pragma unroll
            for (int i = 1; i < kStrips; ++i) v += sums[i][lane];
            a.out[blockIdx.z][s * a.dim + c] = v;
        }
    }
}

bool wide(const NormArgs& a) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.y) |
                          reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.weight);
    return (all & 15u) == 0 && a.dim % 8 == 0 && (a.rows == 1 || (a.ldx % 8 == 0 && a.ldy % 8 == 0 && a.lddy % 8 == 0));
}

template <typename Args>
cudaError_t launch_dependent(void (*kernel)(Args), const Args& a, dim3 grid, int threads, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <bool kF32, bool kWide, int kGroups, bool kWarpRow, int kThreads>
cudaError_t launch(const NormArgs& a, int64_t ctas, cudaStream_t stream) {
    const int threads = kWarpRow ? kThreads : ((a.dim + 8 * kGroups - 1) / (8 * kGroups) + 31) / 32 * 32;
    return launch_dependent(norm_backward_kernel<kF32, kWide, kGroups, kWarpRow, kThreads>, a,
                            dim3(static_cast<unsigned>(ctas), 1, 1), threads, stream);
}

template <bool kF32, bool kWide>
cudaError_t launch(const NormArgs& a, int64_t ctas, cudaStream_t stream) {
    if (a.dim <= 256) return launch<kF32, kWide, 1, true, 256>(a, ctas, stream);
    if (a.dim <= 512) return launch<kF32, kWide, 2, true, 256>(a, ctas, stream);
    if (a.dim <= kNormWarpRowDim) return launch<kF32, kWide, 4, true, 256>(a, ctas, stream);
    if (a.dim <= 4096) return launch<kF32, kWide, 2, false, 256>(a, ctas, stream);
    if (a.dim <= 8192) return launch<kF32, kWide, 2, false, 512>(a, ctas, stream);
    return launch<kF32, kWide, 2, false, 1024>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_norm_backward(const NormArgs& a, bool f32, int64_t ctas, cudaStream_t stream) {
    if (wide(a)) return f32 ? launch<true, true>(a, ctas, stream) : launch<false, true>(a, ctas, stream);
    return f32 ? launch<true, false>(a, ctas, stream) : launch<false, false>(a, ctas, stream);
}

cudaError_t launch_norm_reduce(const NormReduceArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.dim + 31) / 32), static_cast<unsigned>(a.samples < 65535 ? a.samples : 65535),
                    static_cast<unsigned>(a.count));
    return launch_dependent(norm_reduce_kernel, a, grid, 32 * kStrips, stream);
}

}  // namespace mxfp4
