// norm_forward.cu -- layer norm of the rows of X.
//
//   mu = mean(x), r = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) r g + b, g = w or 1 + w,
//   with w and b for the whole of X, for each sample of it (consecutive rows), or not at all.
//
// A row is read once and stays in registers, and its threads meet once.  Each warp centres its part at the mean m_w that
// it finds for it, and gives m_w, the rest r_w = sum(x - m_w) that m_w's rounding left, and
// sum((x - m_w)^2) - r_w^2 / n_w; with d_w = m_w - m_0 + r_w / n_w the row's mean is m_0 + D, D = sum(n_w d_w) / n, and its
// squares are the warps' and n_w (d_w - D)^2.  So nothing is lost where |mu| is far above the deviation.  All of it in
// fp32; y is rounded once.  Bound by the memory, and by instructions not far below it.
//
// A warp takes a short row, a CTA a longer one (launch() below says where).  CTAs stay for many rows, with the
// vectors in registers.  A CTA's rows come through a ring in shared memory, which has three of them on
// their way whatever the registers hold; a warp's are loaded into registers one row ahead.
#include <atomic>

#include "norm_row.cuh"

namespace mxfp4 {
namespace {

template <bool kF32, NormAccess kAccess, int kGroups, RowMode kMode, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) norm_forward_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) uint8_t slots[];
    __shared__ float4 parts[2][32];   // of a row's warps: m, r, squares
    __shared__ RowRing ring;
    using Part = RowPart<kF32, kAccess, kGroups>;
    constexpr bool kWide = Part::kWide;
    constexpr int kP = Part::kPairs, kWarps = kThreads == 320 ? 16 : kThreads / 32;   // of a row's sums: a power of two
    constexpr int kSize = kF32 ? 4 : 2;
    constexpr bool kWarp = kMode == kWarpRow, kRing = kMode == kRingRow;
    const int t = kWarp ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x);
    const int threads = kWarp ? 32 : static_cast<int>(blockDim.x);
    const int64_t stride = kWarp ? static_cast<int64_t>(gridDim.x) * (kThreads / 32) : gridDim.x;   // whole periods, if there is a second row
    int64_t row = kWarp ? static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const int skew = Part::kShifted ? static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const uint8_t*>(a.x) + row * a.ldx * kSize) & 15u) : 0;
    const RowShape shape{a.dim, t, threads, skew / kSize};
    const float inv = 1.0f / static_cast<float>(a.dim);
    const uint8_t* const xs = static_cast<const uint8_t*>(a.x);
    const uint32_t bytes = static_cast<uint32_t>(a.dim) * kSize, slot_bytes = ring_bytes<kWide>(bytes);
    if (kRing) ring_init(&ring, 1, a.stages);
    grid_wait_prerequisites();
    grid_launch_dependents();
    int issued = 0;
    auto copy = [&](int64_t r, int slot) {   // thread 0
        if (*static_cast<volatile int*>(&ring.abort) != 0) return;
        ++issued;
        const uint32_t bar = smem_addr(&ring.full[slot]);
        if (ring_edge<kWide>(r, a.rows)) {
            mbar_arrive(bar);
            return;
        }
        const uint8_t* const from = xs + r * a.ldx * kSize;
        mbar_arrive_expect_tx(bar, ring_moved<kWide>(from, bytes));
        ring_copy<kWide>(smem_addr(slots + slot * slot_bytes), from, bytes, bar);
    };
    if (kRing && threadIdx.x == 0)
        for (int i = 0; i < a.stages && row + i * stride < a.rows; ++i) copy(row + i * stride, i);
    uint64_t g[kP], b[kP];
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        g[i] = both(1.0f);
        b[i] = 0ull;
    }
    // elements of this warp, and of the warp that this lane stands for when the warps' parts are joined
    auto elements = [&](int warp) {
        const RowShape first{a.dim, kWarp ? 0 : 32 * warp, threads, shape.shift};
        int n = 0;
#pragma unroll
        for (int k = 0; k < 2 * kP; k += Part::kTurn) {
            const int c = Part::column(k, first);
            n += max(min(a.dim, c + 32 * Part::kTurn) - max(c, 0), 0);
        }
        return n;
    };
    const int joined = kWarp ? 0 : static_cast<int>(lane_id()) & (kWarps - 1);
    float n_joined = 0.0f, inv_joined = 0.0f;
    if (joined < (kWarp ? 1 : static_cast<int>(blockDim.x >> 5))) {
        n_joined = static_cast<float>(elements(joined));
        inv_joined = n_joined > 0.0f ? 1.0f / n_joined : 0.0f;
    }
    const float inv_own = kWarp ? inv_joined : __shfl_sync(0xFFFFFFFFu, inv_joined, threadIdx.x >> 5);
    int turn = 0;
    int64_t sample = -1;
    Part next;
    if constexpr (!kRing)
        if (row < a.rows) next.load(xs + row * a.ldx * kSize, shape);
    int slot = 0;
    uint32_t phase = 0;
    for (; row < a.rows; row += stride) {
        const int64_t s = row < a.sample_rows ? 0 : row / a.sample_rows;
        if (s != sample) {
            sample = s;
            if (a.weight != nullptr) {
                load_vector<kF32, kAccess, kGroups>(a.weight, s * a.dim, a.w_f32, a.w_wide, shape, g);
                if (a.add_one)
#pragma unroll
                    for (int i = 0; i < kP; ++i) g[i] = add2(g[i], both(1.0f));
            }
            if (a.bias != nullptr) load_vector<kF32, kAccess, kGroups>(a.bias, s * a.dim, a.w_f32, a.w_wide, shape, b);
        }
        if constexpr (kRing) {
            ring_wait(ring, slot, phase, a.err);
            const uint8_t* const from = xs + row * a.ldx * kSize;
            uint8_t* const in = slots + slot * slot_bytes + ring_skew<kWide>(from);
            if (ring_edge<kWide>(row, a.rows)) {
                ring_fill<kF32>(in, from, a.dim, t, threads);
                __syncthreads();
            }
            next.template load<true>(in, shape);
        }
        uint64_t x[kP], sum = 0ull;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            x[i] = next.pair(i);
            sum = add2(sum, x[i]);
        }
        if constexpr (!kRing)
            if (row + stride < a.rows) next.load(xs + (row + stride) * a.ldx * kSize, shape);
        const float2 halves = unpack2(sum);
        float mean = lanes_sum<32>(halves.x + halves.y) * inv_own;
        uint64_t square = 0ull;
        sum = 0ull;
#pragma unroll
        for (int i = 0; i < kP; ++i) x[i] = add2(x[i], Part::kShifted ? both(-mean) : Part::within(-mean, i, shape));
        if constexpr (Part::kShifted) Part::clear(x, shape);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            sum = add2(sum, x[i]);
            square = fma2(x[i], x[i], square);
        }
        const float2 s1 = unpack2(sum), s2 = unpack2(square);
        const float2 own = unpack2(lanes_sum2<32>(pack2(make_float2(s1.x + s1.y, s2.x + s2.y))));
        float shift, var;   // the row's mean less this warp's, and its variance
        if (kWarp) {
            shift = own.x * inv_own;
            var = fmaf(-shift, shift, own.y * inv_own);
        } else {
            if (lane_id() == 0) parts[turn][threadIdx.x >> 5] = make_float4(mean, own.x, own.y, 0.0f);
            __syncthreads();
            if (kRing) {
                if (threadIdx.x == 0 && row + a.stages * stride < a.rows) copy(row + a.stages * stride, slot);
                if (++slot == a.stages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
            const float first = parts[turn][0].x;
            const float4 p = n_joined > 0.0f ? parts[turn][joined] : make_float4(first, 0.0f, 0.0f, 0.0f);
            turn ^= 1;
            const float rest = p.y * inv_joined, d = (p.x - first) + rest;
            const float all = lanes_sum<kWarps>(n_joined * d) * inv, off = d - all;
            var = lanes_sum<kWarps>(fmaf(n_joined * off, off, fmaf(-rest, p.y, p.z))) * inv;
            shift = all - (mean - first);
        }
        mean += shift;
        const float rstd = rsqrtf(fmaxf(var, 0.0f) + a.eps);
        const uint64_t by = both(rstd), less = both(-shift * rstd);
#pragma unroll
        for (int i = 0; i < kP; ++i) x[i] = fma2(fma2(x[i], by, less), g[i], b[i]);
        Part::store(static_cast<uint8_t*>(a.y) + row * a.ldy * kSize, x, shape);
        if (a.mean != nullptr && t == 0) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
    if (kRing && threadIdx.x == 0) ring_drain(ring, a.stages, issued);
}

// kCtas: CTAs that an SM holds at least, by registers.
template <bool kF32, NormAccess kAccess, int kGroups, RowMode kMode, int kThreads, int kCtas>
cudaError_t launch(NormArgs a, int sms, cudaStream_t stream) {
    const auto kernel = norm_forward_kernel<kF32, kAccess, kGroups, kMode, kThreads, kCtas>;
    const int threads = kMode == kWarpRow ? kThreads : row_threads(columns_of(a), kGroups);
    const int64_t need = kMode == kWarpRow ? (a.rows + kThreads / 32 - 1) / (kThreads / 32) : a.rows;
    // The ring: three rows, if they fit beside the CTAs that share the SM.  More CTAs hide more than deeper rings do: 4608 rows of
    // 5120 take 19.9 us with 3 rows, 20.5 with 4, 21.9 with 6, and 26 with 8 in rings that left room for two CTAs.
    constexpr int kBudget = kThreads <= 128 ? 32 * 1024 : kThreads <= 320 ? 64 * 1024 : 192 * 1024;
    const int row_bytes = static_cast<int>(ring_bytes<kAccess == kNormWide>(a.dim * (kF32 ? 4 : 2)));
    a.stages = kMode != kRingRow ? 0 : kBudget / row_bytes < kNormStagesForward ? kBudget / row_bytes : kNormStagesForward;
    const int smem = a.stages * row_bytes;
    // CTAs that an SM holds, by device and warps of the CTA: by registers and threads, and then by the rings
    static std::atomic<int> per_sm[64][kThreads / 32 + 1];
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int>& known = per_sm[dev & 63][threads / 32];
    n = known.load(std::memory_order_relaxed);
    if (n == 0) {
        if (kMode == kRingRow) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBudget);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        known.store(n, std::memory_order_relaxed);
    }
    const int by_rings = kMode == kRingRow ? 227 * 1024 / (smem + 3 * 1024) : n;   // with what a CTA has besides
    const int64_t most = static_cast<int64_t>(n < by_rings ? n : by_rings) * sms;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(need <= most ? need : most / a.period * a.period), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Elements a thread: 32 where rows come in 16-byte accesses, for the join of a row's warps costs each warp as much as
// some 16 elements (8192 rows of 4096: 33 us with 16, 26 with 32; 16384 of 8192: 149 and 88); 16 where they do not, which the
// registers of the single accesses' addresses fill, and 32 again for longer shifted rows (8192 rows of 2500 25 us with 16, 27 with
// 32; of 4001 36 and 32; of 7001 69 and 52).  Single accesses of 4097 to 5120 columns: two CTAs of up to 320 threads an SM, where one of
// the instance for 512 leaves half of it idle (8192 rows of 4100 in fp32 49 us, 69 so; of 5001 55 and 71; 300 of 4500 6.1 and 6.7; bf16
// rows of 4500 whose y is not shifted alike 52 and 72).  A warp's row wins up to 1024 elements: 32768 rows of 1024 take 26 us, 46 as
// a CTA's.  Now 5.3 TB/s at 4096, 6.1 at 8192, 4.7 for 4608 rows of 5120.
template <bool kF32, NormAccess kAccess>
cudaError_t launch(const NormArgs& a, int sms, cudaStream_t stream) {
    const int columns = columns_of(a);
    if constexpr (kAccess != kNormShifted) {
        if (columns <= 256) return launch<kF32, kAccess, 1, kWarpRow, 256, 1>(a, sms, stream);
        if (columns <= kNormWarpRowDim) return launch<kF32, kAccess, 2, kWarpRow, 256, 1>(a, sms, stream);
    }
    if constexpr (kAccess == kNormWide) {
        if (columns <= 1024) return launch<kF32, kAccess, 4, kWarpRow, 128, 4>(a, sms, stream);
        if (columns <= 4096) return launch<kF32, kAccess, 4, kRingRow, 128, 4>(a, sms, stream);
        if (columns <= 8192) return launch<kF32, kAccess, 4, kRingRow, 256, 2>(a, sms, stream);
        return launch<kF32, kAccess, 4, kRingRow, 512, 1>(a, sms, stream);
    } else {
        if (columns <= 2048) return launch<kF32, kAccess, 2, kRingRow, 128, 4>(a, sms, stream);
        if constexpr (kAccess == kNormShifted) {
            if (columns <= 2560) return launch<kF32, kAccess, 2, kRingRow, 256, 2>(a, sms, stream);
            if (columns <= 4096) return launch<kF32, kAccess, 4, kRingRow, 128, 4>(a, sms, stream);
            if (columns <= 8192) return launch<kF32, kAccess, 4, kRingRow, 256, 2>(a, sms, stream);
            return launch<kF32, kAccess, 4, kRingRow, 512, 1>(a, sms, stream);
        } else {
            if (columns <= 4096) return launch<kF32, kAccess, 2, kRingRow, 256, 2>(a, sms, stream);
            if (columns <= 5120) return launch<kF32, kAccess, 2, kRingRow, 320, 2>(a, sms, stream);
            if (columns <= 8192) return launch<kF32, kAccess, 2, kRingRow, 512, 1>(a, sms, stream);
            return launch<kF32, kAccess, 2, kRingRow, 1024, 1>(a, sms, stream);
        }
    }
}

}  // namespace

cudaError_t launch_norm_forward(const NormArgs& a, bool f32, int sms, cudaStream_t stream) {
    if (a.access == kNormWide) return f32 ? launch<true, kNormWide>(a, sms, stream) : launch<false, kNormWide>(a, sms, stream);
    if (a.access == kNormShifted) return launch<false, kNormShifted>(a, sms, stream);
    return f32 ? launch<true, kNormSingle>(a, sms, stream) : launch<false, kNormSingle>(a, sms, stream);
}

}  // namespace mxfp4
