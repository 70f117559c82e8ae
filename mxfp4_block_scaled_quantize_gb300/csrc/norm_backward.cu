// norm_backward.cu -- the backward pass of layer norm, with the gradients of its weight and bias.
//
// With xh = (x - mu) r and a = dy g (g = w or 1 + w):
//   dx = r (a - mean(a) - xh mean(a xh)),  dw = sum over rows of dy xh,  db = sum over rows of dy.
//
// One pass over X and dY: a CTA takes a range of consecutive rows of one sample (rows of up to 512
// elements: a warp each), keeps its columns' sums of dw and db in registers across them, and
// leaves them as one partial row; a second kernel adds the partial rows in a fixed order, so the same
// inputs give the same bits.  A sample that is one CTA's needs no second kernel.  Rows come as in the
// forward pass, x and dy side by side in a slot of the ring.  Bound by the memory: x and dy in, dx
// out; the partial rows are 4 / chunk_rows of x and dy in bf16.
//
// 16 elements a thread, for dw, db and the gain in registers leave room for no more at 512 threads an SM (8 a thread and 1024
// threads: 16384 rows of 8192 in 156 us, 129 with 16; 24 warps at 85 registers each spill: 8192 of 4096 in 58 us, 40 with 16 warps;
// two teams of rows of 5120 have it in shared memory).
// Now 6.2 TB/s for 16384 rows of 8192, 5.3 for 8192 of 4096, of whose 38 us the partial rows and the second kernel take 6.  Rows of more
// than 8192 elements have 64 registers a thread, and spill: 4096 rows of 16384 take 187 us, 2.2 TB/s.
#include <atomic>

#include "norm_row.cuh"

namespace mxfp4 {
namespace {

// A CTA of shorter rows has teams of kThreads threads at most, 512 in all, each with a row and a ring to itself, and one partial row for
// all of them.  (As a CTA each: 8192 rows of 4096 39.7 us, 38 so; 8192 of 1001 24.8 and 20.4; 1111 of 1001 11.9 and 9.0.)
template <RowMode kMode, int kThreads>
constexpr int kTeamsOf = kMode != kRingRow ? 1 : kThreads == 320 ? 2 : kThreads < 512 ? 512 / kThreads : 1;

// Two teams of 320 threads have 96 registers each: their gains are in shared memory, where each thread finds its own.
template <int kThreads>
constexpr bool kGainsStored = kThreads == 320;

template <bool kF32, NormAccess kAccess, int kGroups, RowMode kMode, int kThreads, int kCtas>
__global__ void __launch_bounds__(kThreads * kTeamsOf<kMode, kThreads>, kCtas) norm_backward_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ __align__(16) uint8_t shared_bytes[];
    using Part = RowPart<kF32, kAccess, kGroups>;
    constexpr bool kWide = Part::kWide;
    constexpr int kE = Part::kElements, kP = Part::kPairs;
    constexpr int kSize = kF32 ? 4 : 2;
    constexpr int kWarps = kThreads == 320 ? 16 : kThreads / 32;   // of a row's sums: a power of two
    constexpr bool kWarp = kMode == kWarpRow, kRing = kMode == kRingRow;
    constexpr int kTeams = kTeamsOf<kMode, kThreads>;
    __shared__ uint64_t team_sums[kTeams][2][kWarps];
    __shared__ RowRing rings[kTeams];
    __shared__ float sums[kWarp ? kWarps : 1][kWarp ? 32 * kE : 1];
    const int threads = kWarp ? 32 : static_cast<int>(blockDim.x) / kTeams;
    const int team = kTeams > 1 ? static_cast<int>(threadIdx.x) / threads : 0;
    const int t = kWarp ? static_cast<int>(lane_id()) : static_cast<int>(threadIdx.x) - team * threads;
    RowRing& ring = rings[team];
    // rows first, first + period, ..., chunk_rows of them at most
    const int64_t sample = blockIdx.x / a.chunks;
    const int32_t chunk = blockIdx.x % a.chunks;
    const int64_t in_sample = chunk % a.period + static_cast<int64_t>(chunk / a.period) * a.chunk_rows * a.period;
    const int64_t first = sample * a.sample_rows + in_sample;
    const int64_t end = sample * a.sample_rows + min(in_sample + a.chunk_rows * a.period, a.sample_rows);
    const int64_t stride = (kWarp ? kWarps : kTeams) * static_cast<int64_t>(a.period);
    const int skew = Part::kShifted ? static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const uint8_t*>(a.x) + first * a.ldx * kSize) & 15u) : 0;
    const RowShape shape{a.dim, t, threads, skew / kSize};
    const float inv = 1.0f / static_cast<float>(a.dim);
    const uint8_t *const xs = static_cast<const uint8_t*>(a.x), *const ys = static_cast<const uint8_t*>(a.dy);
    const uint32_t bytes = static_cast<uint32_t>(a.dim) * kSize, part_bytes = ring_bytes<kWide>(bytes);
    uint8_t* const slots = shared_bytes + (kRing ? 2 * team * a.stages * part_bytes : 0u);
    if (kRing) ring_init(rings, kTeams, a.stages);
    grid_wait_prerequisites();
    grid_launch_dependents();
    int64_t row = first + (kWarp ? static_cast<int64_t>(threadIdx.x >> 5) : static_cast<int64_t>(team)) * a.period;
    int issued = 0;   // of a team's thread 0: the copies so far
    auto copy = [&](int64_t r, int slot) {   // one thread
        if (*static_cast<volatile int*>(&ring.abort) != 0) return;
        ++issued;
        const uint32_t bar = smem_addr(&ring.full[slot]), to = smem_addr(slots + 2 * slot * part_bytes);
        if (ring_edge<kWide>(r, a.rows)) {
            mbar_arrive(bar);
            return;
        }
        const uint8_t *const x = xs + r * a.ldx * kSize, *const y = ys + r * a.lddy * kSize;
        mbar_arrive_expect_tx(bar, ring_moved<kWide>(x, bytes) + ring_moved<kWide>(y, bytes));
        ring_copy<kWide>(to, x, bytes, bar);
        ring_copy<kWide>(to + part_bytes, y, bytes, bar);
    };
    if (kRing && lane_id() == 0) {   // the first rows, each by another warp: a copy costs its thread some 400 clocks
        for (int i = t >> 5; i < a.stages && row + i * stride < end; i += threads >> 5) copy(row + i * stride, i);
        issued = 0;
        while (issued < a.stages && row + issued * stride < end) ++issued;
    }
    uint64_t g[kP], dw[kP], db[kP];
    ulonglong2* const gains = reinterpret_cast<ulonglong2*>(shared_bytes + (kRing ? 2 * kTeams * a.stages * part_bytes : 0u)) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
        g[i] = both(1.0f);
        dw[i] = 0ull;
        db[i] = 0ull;
    }
    if (a.weight != nullptr) {
        load_vector<kF32, kAccess, kGroups>(a.weight, sample * a.dim, a.w_f32, a.w_wide, shape, g);
        if (a.add_one)
#pragma unroll
            for (int i = 0; i < kP; ++i) g[i] = add2(g[i], both(1.0f));
    }
    if constexpr (kGainsStored<kThreads>)
#pragma unroll
        for (int i = 0; i < kP; i += 2) gains[i / 2 * kTeams * kThreads] = make_ulonglong2(g[i], g[i + 1]);
    Part nx, ny;
    float nmean = 0.0f, nrstd = 0.0f;
    auto fetch = [&](int64_t r) {
        if constexpr (!kRing) {
            nx.load(xs + r * a.ldx * kSize, shape);
            ny.load(ys + r * a.lddy * kSize, shape);
        }
        nmean = __ldg(a.mean + r);
        nrstd = __ldg(a.rstd + r);
    };
    if (row < end) fetch(row);
    int turn = 0, slot = 0;
    uint32_t phase = 0;
    for (; row < end; row += stride, turn ^= 1) {
        if constexpr (kRing) {
            ring_wait(ring, slot, phase, a.err);
            const uint8_t *const x = xs + row * a.ldx * kSize, *const y = ys + row * a.lddy * kSize;
            uint8_t* const in = slots + 2 * slot * part_bytes;
            if (ring_edge<kWide>(row, a.rows)) {
                ring_fill<kF32>(in + ring_skew<kWide>(x), x, a.dim, t, threads);
                ring_fill<kF32>(in + part_bytes + ring_skew<kWide>(y), y, a.dim, t, threads);
                row_meet<(kTeams > 1)>(team, threads);
            }
            nx.template load<true>(in + ring_skew<kWide>(x), shape);
            ny.template load<true>(in + part_bytes + ring_skew<kWide>(y), shape);
        }
        const float mean = nmean, rstd = nrstd;
        uint64_t xh[kP], c[kP], sa = 0ull, sx = 0ull;
#pragma unroll
        for (int i = 0; i < kP; ++i) {   // dy is zero behind the row's end
            if constexpr (kGainsStored<kThreads>)
                if (i % 2 == 0) {
                    const ulonglong2 v = gains[i / 2 * kTeams * kThreads];
                    g[i] = v.x;
                    g[i + 1] = v.y;
                }
            const uint64_t d = ny.pair(i);
            xh[i] = mul2(add2(nx.pair(i), both(-mean)), both(rstd));
            c[i] = mul2(d, g[i]);
            dw[i] = fma2(d, xh[i], dw[i]);
            db[i] = add2(db[i], d);
            sa = add2(sa, c[i]);
            sx = fma2(c[i], xh[i], sx);
        }
        if (row + stride < end) fetch(row + stride);
        const float2 s1 = unpack2(sa), s2 = unpack2(sx);
        const float2 sum = row_sum2<kMode, kWarps, (kTeams > 1)>(pack2(make_float2(s1.x + s1.y, s2.x + s2.y)), team_sums[team][turn], t, team, threads);
        if (kRing) {
            if (t == 0 && row + a.stages * stride < end) copy(row + a.stages * stride, slot);
            if (++slot == a.stages) {
                slot = 0;
                phase ^= 1u;
            }
        }
        const uint64_t m1 = both(-sum.x * inv), m2 = both(-sum.y * inv);
#pragma unroll
        for (int i = 0; i < kP; ++i) c[i] = mul2(add2(fma2(xh[i], m2, c[i]), m1), both(rstd));
        Part::store(static_cast<uint8_t*>(a.y) + row * a.ldy * kSize, c, shape);
    }
    if (kRing && t == 0) ring_drain(ring, a.stages, issued);
    if constexpr (kTeams > 1) {
        if (a.partial_w == nullptr && a.partial_b == nullptr) return;
        // The teams' rows in the rings' place: 2 kTeams of fp32, where each team had room for two rows of fp32 or four of bf16 at least.
        float* const rows = reinterpret_cast<float*>(shared_bytes);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float* const out = rows + (i * kTeams + team) * a.dim;
            const uint64_t* const v = i == 0 ? dw : db;
            if constexpr (kWide) {
                RowPart<true, kNormWide, kGroups>::store(out, v, shape);
            } else {
#pragma unroll
                for (int k = 0; k < kP; ++k) {
                    const float2 f = unpack2(v[k]);
                    if (Part::inside(2 * k, shape)) out[Part::column(2 * k, shape)] = f.x;
                    if (Part::inside(2 * k + 1, shape)) out[Part::column(2 * k + 1, shape)] = f.y;
                }
            }
        }
        __syncthreads();
        for (int i = 0; i < 2; ++i) {
            float* const to = i == 0 ? a.partial_w : a.partial_b;
            if (to == nullptr) continue;
            for (int c = threadIdx.x; c < a.dim; c += blockDim.x) {
                float s = 0.0f;
#pragma unroll
                for (int j = 0; j < kTeams; ++j) s += rows[(i * kTeams + j) * a.dim + c];
                to[static_cast<int64_t>(blockIdx.x) * a.dim + c] = s;
            }
        }
        return;
    }
    float* const to[2] = {a.partial_w, a.partial_b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (to[i] == nullptr) continue;
        float* const out = to[i] + static_cast<int64_t>(blockIdx.x) * a.dim;
        const uint64_t* const v = i == 0 ? dw : db;
        if (kWarp) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kP; ++k) {
                const float2 f = unpack2(v[k]);
                sums[threadIdx.x >> 5][Part::column(2 * k, shape)] = f.x;
                sums[threadIdx.x >> 5][Part::column(2 * k + 1, shape)] = f.y;
            }
            __syncthreads();
            for (int c = threadIdx.x; c < a.dim; c += kThreads) {
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += sums[w][c];
                out[c] = s;
            }
        } else if (kWide && (reinterpret_cast<uintptr_t>(out) & 15u) == 0) {
            RowPart<true, kNormWide, kGroups>::store(out, v, shape);
        } else {
#pragma unroll
            for (int k = 0; k < kP; ++k) {
                const float2 f = unpack2(v[k]);
                if (Part::inside(2 * k, shape)) out[Part::column(2 * k, shape)] = f.x;
                if (Part::inside(2 * k + 1, shape)) out[Part::column(2 * k + 1, shape)] = f.y;
            }
        }
    }
}

// Sums of the partial rows: 32 columns of one sample a CTA, 32 strips of its partial rows.
constexpr int kStrips = 32;
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
#pragma unroll 10
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

template <typename Args>
cudaError_t launch_dependent(void (*kernel)(Args), const Args& a, dim3 grid, int threads, int smem, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// kCtas: CTAs that an SM holds, by registers.
template <bool kF32, NormAccess kAccess, int kGroups, RowMode kMode, int kThreads, int kCtas>
cudaError_t launch(NormArgs a, int64_t ctas, cudaStream_t stream) {
    const auto kernel = norm_backward_kernel<kF32, kAccess, kGroups, kMode, kThreads, kCtas>;
    const int threads = kMode == kWarpRow ? kThreads : row_threads(columns_of(a), kGroups);
    // The ring: as many rows as fit beside the CTAs that share the SM.
    constexpr int kTeams = kTeamsOf<kMode, kThreads>, kGainBytes = kGainsStored<kThreads> ? 32 * kGroups * kTeams * kThreads : 0;
    constexpr int kBudget = (208 * 1024 - kGainBytes) / kTeams;   // of a team: what is left is for the rest
    const int slot_bytes = 2 * static_cast<int>(ring_bytes<kAccess == kNormWide>(a.dim * (kF32 ? 4 : 2)));
    a.stages = kMode != kRingRow ? 0 : kBudget / slot_bytes < kNormStagesBackward ? kBudget / slot_bytes : kNormStagesBackward;
    if (kMode == kRingRow) {   // once a device: the call costs the host as much as a launch
        static std::atomic<uint64_t> known{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = uint64_t{1} << (dev & 63);
        if (!(known.load(std::memory_order_relaxed) & bit)) {
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTeams * kBudget + kGainBytes);
            if (e != cudaSuccess) return e;
            known.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    return launch_dependent(kernel, a, dim3(static_cast<unsigned>(ctas), 1, 1), kTeams * threads, kTeams * a.stages * slot_bytes + kGainBytes, stream);
}

// Two teams for rows of 4097 to 5120 elements, in place of one that leaves a third of the SM's registers, pay where a CTA has many
// rows: 16384 rows of 4608 84 us, 96 with one; 9000 of 4200 50 and 56; 16384 of 5120 93 and 98; 8192 of 5120 in fp32 90 and 93; but 4608 of
// 5120 35.7 and 35.4, 2048 of 5120 22.4 and 21.5, 4096 of 4608 in fp32 44.6 and 42.0.
template <bool kF32, NormAccess kAccess>
cudaError_t launch(const NormArgs& a, int64_t ctas, cudaStream_t stream) {
    const int columns = columns_of(a);
    if constexpr (kAccess != kNormShifted) {
        if (columns <= 256) return launch<kF32, kAccess, 1, kWarpRow, 256, 2>(a, ctas, stream);
        if (columns <= kNormWarpRowDim) return launch<kF32, kAccess, 2, kWarpRow, 256, 2>(a, ctas, stream);
    }
    if (columns <= 1024) return launch<kF32, kAccess, 2, kRingRow, 64, 1>(a, ctas, stream);
    if (columns <= 2048) return launch<kF32, kAccess, 2, kRingRow, 128, 1>(a, ctas, stream);
    if (columns <= 4096) return launch<kF32, kAccess, 2, kRingRow, 256, 1>(a, ctas, stream);
    if constexpr (kAccess == kNormWide)
        if (columns <= 5120 && a.chunk_rows >= 32) return launch<kF32, kAccess, 2, kRingRow, 320, 1>(a, ctas, stream);
    if (columns <= 8192) return launch<kF32, kAccess, 2, kRingRow, 512, 1>(a, ctas, stream);
    return launch<kF32, kAccess, 2, kRingRow, 1024, 1>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_norm_backward(const NormArgs& a, bool f32, int64_t ctas, cudaStream_t stream) {
    if (a.access == kNormWide) return f32 ? launch<true, kNormWide>(a, ctas, stream) : launch<false, kNormWide>(a, ctas, stream);
    if (a.access == kNormShifted) return launch<false, kNormShifted>(a, ctas, stream);
    return f32 ? launch<true, kNormSingle>(a, ctas, stream) : launch<false, kNormSingle>(a, ctas, stream);
}

cudaError_t launch_norm_reduce(const NormReduceArgs& a, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((a.dim + 31) / 32), static_cast<unsigned>(a.samples < 65535 ? a.samples : 65535),
                    static_cast<unsigned>(a.count));
    return launch_dependent(norm_reduce_kernel, a, grid, 32 * kStrips, 0, stream);
}

}  // namespace mxfp4
