// experts.cu -- a whole mixture-of-experts layer for a few tokens, in one kernel.
//
//   p = softmax(logits), the top_k largest of them (ties: the lowest index), w = p or p / sum of the chosen p,
//   y_t = sum over the chosen experts e of w_e W2_e . (silu(g) u),   [g; u] = W1_e . x_t,   silu(g) = g / (1 + exp(-g)),
//   W1 [E, 2 inner, dim], W2 [E, dim, inner] in MXFP4 (E2M1 codes, an E8M0 scale for 32 along the row).
//
// For a few tokens the time is that of the chosen experts' weights, each read once: 17 / 32 bytes an element at 23 bytes a
// clock and SM.  So the activations stay as they are (rounding them to 4 bits would save nothing), and a product has the
// weights as the 16 rows of a small matrix instruction (mma.sync m16n8k16; the tcgen05 forms would want 128 rows of one
// expert and 4-bit or 8-bit activations) and up to 16 routed rows as its columns.
//
// Numbers.  A code is exact in fp16.  x is bf16 times a power of two that brings its row's largest value to 2^14 .. 2^15: exact
// in fp16 but for what lies more than 2^-31 below it, which is off by 2^-39 of it at most (half of fp16's smallest step).  The activations
// between the products are fp32, and the second product takes them as the sum of two fp16 (22 bits).  A block of 32 is summed by
// the matrix instruction in fp32 and then multiplied by its scale in fp32, as all sums are; the power of two is undone after
// them: k elements of codes up to 6 stay below k 6 2^15 times the scale, in fp32's range up to a scale of 2^96 for every k that
// fits the shared memory.  y is rounded once.
//
// Four phases, with the grid meeting in between (a cooperative launch, one CTA an SM; a barrier takes 1 to 2 us):
//   1. CTA t: token t's choices, and its row of x in fp16.  (Up to kFew tokens: every CTA, all of them, and no barrier.)
//   2. The first product, with silu(g) u.   3. The second product.   4. The sums over the experts, in the tokens' order.
// (As two kernels that each routed and staged for themselves, and with the sums left to whichever CTA came last for 32
// columns: 137 us where one kernel then took 115, of which 60 passed before the first and after the last weights.)
//
// Work of phases 2 and 3.  A unit is 32 rows of an expert's weights (16 of g and the same 16 of u) against a pass of its routed
// rows.  A CTA takes a range of consecutive units, so it stages an expert's activations in shared memory once.  Its 16 warps
// take 16 units of one expert at a time, a whole unit each, and meet nobody; the n < 16 that are left they share, each with
// 1 / 16 of all their slices of 128 elements, which are of two units at most: a unit's first warp adds what the others found.
// (All units dealt out slice by slice to 16 warps, which met after each one, took 1.9 times the instructions; the rest in
// rounds of 8, 4, 2 and 1 units 9 us more in some CTAs than in others, of 50.)  Each warp has several slices (2 KB of codes) on
// their way to shared memory by copies of its own, across the ends of its units and, to the second product's weights, across the barrier.
//   The order of all additions is fixed by the call's routing.
//   (The two fp16 of an activation between the products cost a second set of matrix instructions: 17 us of the 209 for 64 tokens
// below.  Up to 4 rows have them side by side as 8 columns, which costs none: 8 tokens 59 us, 65 without that.)
//
// Both products go through the same code.  (Written out for each, with what a product multiplies as constants, it took as long.)
//
// Measured (experts dim x inner; 1, 8 and 32 tokens of 8 of 64, 2048 x 1408; 64 of 6 of 64, 4096 x 2048): 26, 59, 85 and 206 us,
// where the weights' bytes take 5.4, 28.5, 42.8 and 126.  One token: 2 us for the choices, 1.5 for the lists, 1.7 until the first weights
// are asked for, 6.2 for the first product, 4.8 for the second, 5 for the two barriers and the sums, and 4 before and after.
// 64 tokens: the first product at 20 bytes a clock and SM (of 23), the second at 16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "launch.h"
#include "launch_experts.h"
#include "ptx.cuh"

namespace mxfp4 {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kUnitRows = 32;
constexpr int kSlice = 128;                              // elements of a row
constexpr int kSliceBytes = kUnitRows * kSlice / 2;      // codes
constexpr int kWordBytes = 4 * kUnitRows;                // and a word of four scales for each row
constexpr int kMaxStages = 4;
constexpr int kMaxPass = 16;                             // routed rows of a pass
// Up to kFew tokens, every CTA chooses for all of them and stages them by itself, and needs no barrier for it: one token 26 us, 28
// with the barrier; 4 take 46 either way, and 8 a little more without it, for a warp then has a row to itself.
constexpr int kFew = 4;
constexpr int kSharedMost = 227 * 1024;
// A unit of a pass of more than 8 rows takes 1.6 times as long as one of up to 8, and coming to another expert or pass as long as
// kStagingSlices slices of a unit (32 tokens, 8 of 64: 88 us without counting that, 84.6 with 32 slices, 83.3 with 64, 82.2 with 96;
// 8 tokens: 64.9, 60.8, 61.4, 63.1).
constexpr uint32_t kNarrowCost = 5, kWideCost = 8, kStagingSlices = 64;

struct Row {           // of a pass
    int32_t slot;      // token * top_k + place among the token's choices; -1: no row
    float back;        // undoes the power of two of its activations
    float weight;
    uint32_t from;     // its activations' row
};

// Shared memory: this head, then [experts] masks, [tokens * top_k] weights, what undoes the activations' powers of two (of a
// token, then of a choice) and experts, the list of (expert, pass),
// the activations, the units' sums, the warps' scales, their words and (at a multiple of 512 bytes) their codes.
struct Head {
    Row rows[kMaxPass];
    int32_t range[4];  // the CTA's units of the first product: from, to; of the second
    int32_t narrow;    // (expert, pass) pairs of up to 8 rows
    int32_t wide;      // the pass has more than 8 rows,
    int32_t slim;      // up to 4: the second product then has its activations' low parts beside the high ones, as columns 4 to 7
    int32_t abort;     // a wait has run out
    int32_t lost[kWarps];  // of a warp whose first lane gave a wait up: 1 + 2 times the stage + 256 times the parity that it waited for; else 0
    uint32_t tops[kFew];   // largest magnitudes of rows of x, as bits
    uint64_t full[kWarps][kMaxStages];
};

__host__ __device__ inline int align16(int n) { return (n + 15) & ~15; }

// n / d for n d < 2^32, by = 2^32 / d rounded up, or 0 for d = 1.  (A division is 30 instructions, most of them waiting for one another.)
__device__ __forceinline__ int divide(int n, uint32_t by) { return by == 0u ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), by)); }

struct Layout {
    int masks, weights, backs, ids, list, list_size, acts, sums, scales, words, codes, total;
    __host__ __device__ Layout(int experts, int tokens, int top_k, int dim, int inner, int pass_rows, int stage_count) {
        const int choices = tokens * top_k, up = pass_rows * pitch(dim), down = 2 * pass_rows * pitch(inner);
        masks = align16(sizeof(Head));
        weights = masks + align16(8 * experts);
        backs = weights + align16(4 * choices);
        ids = backs + align16(4 * choices);
        list = ids + align16(2 * choices);
        // an expert's passes: one, and one more for every further pass_rows of its tokens
        list_size = (experts < choices ? experts : choices) + choices / pass_rows;
        acts = list + align16(4 * list_size);
        sums = acts + (up > down ? up : down);
        scales = sums + kWarps * kUnitRows * pass_rows * 4;
        words = scales + kWarps * kUnitRows * 16;
        codes = (words + kWarps * stage_count * kWordBytes + 511) & ~511;
        total = codes + kWarps * stage_count * kSliceBytes;
    }
    // Bytes from one row of the activations to the next: 64 more than a multiple of 128, so that the 16-byte
    // loads of two rows' four lanes each meet all banks once.
    __host__ __device__ static int pitch(int k) { return 2 * ((k + kSlice - 1) / kSlice * kSlice) + 64; }
};

// Of the 16 (4) bytes that these write, the first `bytes` are read, the others zero.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
// This thread's copies so far arrive at the barrier, as one of its expected arrivals, when they are done.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most kLeft of this thread's groups are under way.
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// Eight codes as four pairs of fp16.
__device__ __forceinline__ void decode8(uint32_t w, uint32_t* h) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Words (row lane / 4, word lane % 4) of four matrices of 8 rows of 16 bytes; lane l brings the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void load_words4(uint32_t* w, uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at)
                 : "memory");
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 2^(byte - 127) for byte b of w, as bits.
__device__ __forceinline__ uint32_t scale_of(uint32_t w, int b) {
    return max((b < 3 ? w << (23 - 8 * b) : w >> 1) & 0x7F800000u, 0x00400000u);
}

__device__ __forceinline__ uint32_t max_all(uint32_t v) {
    uint32_t m;
    asm volatile("redux.sync.max.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(v));
    return m;
}
__device__ __forceinline__ uint32_t min_all(uint32_t v) {
    uint32_t m;
    asm volatile("redux.sync.min.u32 %0, %1, 0xffffffff;" : "=r"(m) : "r"(v));
    return m;
}
__device__ __forceinline__ float sum_all(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

__device__ __forceinline__ float logit_of(const ExpertsArgs& a, int64_t t, int e) {
    const int64_t i = t * a.ldl + e;
    return a.logits_f32 ? __ldcg(static_cast<const float*>(a.logits) + i)
                        : __uint_as_float(static_cast<uint32_t>(__ldcg(static_cast<const uint16_t*>(a.logits) + i)) << 16);
}

// Phase 1 for one token, by one warp: its choices and their weights.  kPer: 32 kPer experts at most.  Order: value, then lowest
// index; a NaN is above all values, as in a sort.
template <int kPer>
__device__ __forceinline__ void choose(const ExpertsArgs& a, int t, float* weights, uint16_t* ids) {
    const int lane = static_cast<int>(lane_id());
    const float none = __int_as_float(0xFF800000);
    float v[kPer];
    uint32_t key[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = i * 32 + lane;
        v[i] = e < a.experts ? logit_of(a, t, e) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const uint32_t u = __float_as_uint(v[i] + 0.0f);   // one zero
        key[i] = v[i] != v[i] ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
        if (i * 32 + lane >= a.experts) key[i] = 0u;       // below every value
    }
    float mine = 0.0f, top = 0.0f;   // lane j: the value of choice j
    int id = 0;
#pragma unroll 1
    for (int j = 0; j < a.top_k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t most = max_all(best);
        const int e = static_cast<int>(min_all(best == most ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu));
        float value = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i * 32 + lane == e) {
                key[i] = 0u;
                value = v[i];
            }
        value = __shfl_sync(0xFFFFFFFFu, value, e & 31);
        if (j == 0) top = value;
        if (lane == j) {
            mine = value;
            id = e;
        }
    }
    const float p = lane < a.top_k && mine != none ? expf(mine - top) : 0.0f;
    float sum = p;
    if (!a.normalize) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (i * 32 + lane < a.experts && v[i] != none) sum += expf(v[i] - top);
    }
    sum = sum_all(sum);
    if (lane < a.top_k) {
        weights[t * a.top_k + lane] = sum == 0.0f ? 0.0f : p / sum;   // 0: every logit is -inf
        ids[t * a.top_k + lane] = static_cast<uint16_t>(id);
    }
}
__device__ __forceinline__ void choose(const ExpertsArgs& a, int t, float* weights, uint16_t* ids) {
    if (a.experts <= 64) choose<2>(a, t, weights, ids);
    else if (a.experts <= 256) choose<8>(a, t, weights, ids);
    else choose<32>(a, t, weights, ids);
}

// 2^k that brings `top` to 2^14 .. 2^15 (k <= 126), and 2^-k.
__device__ __forceinline__ float lift(float top, float* back) {
    const int e = static_cast<int>(__float_as_uint(top) >> 23);   // of a finite value >= 0
    const int k = e == 0 ? 126 : min(14 - (e - 127), 126);
    *back = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    return __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
}

__device__ __forceinline__ float finite_or_zero(float v) {
    v = fabsf(v);
    return v < __int_as_float(0x7F800000) ? v : 0.0f;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight elements of x's row from c on.
__device__ __forceinline__ void x8(const ExpertsArgs& a, const uint16_t* row, int c, bool wide, float* f) {
    if (wide && c < a.dim) {
        const uint4 u = *reinterpret_cast<const uint4*>(row + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < a.dim ? __uint_as_float(static_cast<uint32_t>(row[c + i]) << 16) : 0.0f;
}

// Token t's row of x in fp16, zeros behind its end, by `threads` threads (whole warps) of which this is number `first`; to: its
// place, back: that of what undoes the row's power of two.  `barrier` is theirs, or also others' who come to it as often.
__device__ __forceinline__ void lower_row(const ExpertsArgs& a, int t, int first, int threads, uint32_t* head_top, uint32_t barrier_threads, uint4* to,
                                          float* back_to) {
    const uint16_t* const row = a.x + t * a.ldx;
    const bool wide = a.dim % 8 == 0 && (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    const int groups = (Layout::pitch(a.dim) - 64) / 16;
    float top = 0.0f;
#pragma unroll 1
    for (int i = first; wide && i < groups; i += 8 * threads) {
        uint4 u[8];   // on their way together
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = 8 * (i + j * threads);
            u[j] = c < a.dim ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(finite_or_zero(__uint_as_float(w[k] << 16)), finite_or_zero(__uint_as_float(w[k] & 0xFFFF0000u))));
#pragma unroll
            for (int k = 0; k < 7; ++k) u[k] = u[k + 1];
        }
    }
#pragma unroll 1
    for (int i = first; !wide && i < groups; i += threads) {
        float f[8];
        x8(a, row, 8 * i, false, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_or_zero(f[j]));
    }
    const uint32_t most = max_all(__float_as_uint(top));
    if (lane_id() == 0) atomicMax(head_top, most);   // the order does not matter
    named_barrier(1, barrier_threads);
    float back;
    const float up = lift(__uint_as_float(*head_top), &back);
    if (first == 0) *back_to = back;
#pragma unroll 1
    for (int i = first; i < groups; i += threads) {
        float f[8];
        x8(a, row, 8 * i, wide, f);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = half2_of(f[2 * j] * up, f[2 * j + 1] * up);
        to[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// The grid meets: what every thread wrote before is there for every thread after.  A wait that runs out is recorded, and
// the CTA goes on: no CTA is left waiting for good.
__device__ __forceinline__ void meet(const ExpertsArgs& a, int which) {
    __syncthreads();
    if (threadIdx.x == 0) {
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(&a.sync->arrived[which]) : "memory");   // the CTA's writes before
        const uint64_t t0 = globaltimer();
        for (;;) {
            uint32_t n = 0;
#pragma unroll 1
            for (int i = 0; i < 64; ++i) {
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(&a.sync->arrived[which]) : "memory");
                if (n >= gridDim.x) break;
            }
            if (n >= gridDim.x) break;
            if (globaltimer() - t0 > kWaitLimitNs) {
                atomicOr(a.err, kErrExperts);
                break;
            }
        }
    }
    __syncthreads();
}

// The unit at which CTA `cta` starts, so that all have the same to do.
__device__ __forceinline__ int range_start(const ExpertsSide& side, uint32_t narrow, uint32_t wide, uint32_t cta) {
    const uint32_t tiles = static_cast<uint32_t>(side.tiles), slices = static_cast<uint32_t>(side.slices);
    // of a unit, of a pair; all of it is below 2^30: at most 1200 pairs of 300 units of 74 slices
    const uint32_t unit_n = kNarrowCost * slices, unit_w = kWideCost * slices;
    const uint32_t staging = kNarrowCost * kStagingSlices;
    const uint32_t pair_n = tiles * unit_n + staging, pair_w = tiles * unit_w + staging;
    const uint32_t all = narrow * pair_n + wide * pair_w, share = all / gridDim.x;
    uint32_t at = share * cta + (all - share * gridDim.x) * cta / gridDim.x, first = 0, pair = pair_n, unit = unit_n;
    if (at >= narrow * pair_n) {
        at -= narrow * pair_n;
        first = narrow;
        pair = pair_w;
        unit = unit_w;
    }
    const uint32_t p = at / pair, in = at - p * pair;
    return static_cast<int>((first + p) * tiles + (in <= staging ? 0 : (in - staging) / unit));
}

// Each expert's tokens, and the list of (expert, pass) pairs that have any: those of up to 8 rows from its front on, the
// others from its back on.  The masks are zero before.
__device__ __forceinline__ void list_pairs(const ExpertsArgs& a, Head* head, unsigned long long* masks, float* weights, uint16_t* ids, uint32_t* list,
                                           int list_size, float* backs) {
    const bool here = a.tokens <= kFew;   // this CTA's own choices are there already
#pragma unroll 1
    for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads) {
        float w;
        int e;
        if (here) {
            w = weights[i];
            e = ids[i];
        } else {
            weights[i] = w = __ldcg(a.weights + i);
            ids[i] = static_cast<uint16_t>(e = min(static_cast<int>(__ldcg(a.ids + i)), a.experts - 1));   // a barrier that gave up may have left anything there
        }
        if (w != 0.0f) atomicOr(&masks[e], 1ull << (i / a.top_k));   // not where it changes nothing
    }
    if (!here && threadIdx.x < a.tokens) backs[threadIdx.x] = __ldcg(a.backs + threadIdx.x);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = static_cast<int>(lane_id());
        int before = 0;   // pairs of the experts before: narrow ones, and 2^16 times the wide ones
#pragma unroll 1
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < a.experts ? __popcll(masks[e]) : 0;
            const int full = a.passes_rows > 8 ? n >> 4 : n >> 3, rest = n & (a.passes_rows - 1);
            const int wide = a.passes_rows > 8 ? full + (rest > 8) : 0;
            const int mine = (full + (rest > 0) - wide) | wide << 16;
            int sum = mine;   // inclusive over the lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += up;
            }
            int at = before + sum - mine;
#pragma unroll 1
            for (int p = 0; p < full + (rest > 0); ++p) {
                const bool is_wide = p < wide;   // full passes first, the one with the rest last
                list[is_wide ? list_size - 1 - (at >> 16) : at & 0xFFFF] = static_cast<uint32_t>(e) | static_cast<uint32_t>(p) << 16;
                at += is_wide ? 1 << 16 : 1;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        const uint32_t narrow = static_cast<uint32_t>(before & 0xFFFF), wide = static_cast<uint32_t>(before >> 16);
        if (lane == 0) head->narrow = static_cast<int32_t>(narrow);
        if (lane < 4) head->range[lane] = range_start(a.side[lane >> 1], narrow, wide, blockIdx.x + (lane & 1));
    }
    __syncthreads();
}

// Pair p of the list, those of up to 8 rows first.
struct Pairs {
    const uint32_t* list;
    int size, narrow;
    __device__ __forceinline__ uint32_t operator[](int p) const { return list[p < narrow ? p : size - 1 - (p - narrow)]; }
};

// A warp's way through the CTA's units, one segment (slices of one unit) after the other.  Rounds of 16 units of one expert and
// pass have one for each warp, a whole unit.  A round of the n < 16 that are left has two: the warp's share of the n units'
// slices, first what it has of a unit that another warp begins, then what it begins itself; either may be empty.
struct Segments {
    enum Kind { kWhole, kGoOn, kBegin };
    int end, warp;
    int base, next;        // the round's first unit, and the next round's
    int pair;              // its place in the list of (expert, pass)
    int left;              // its units
    int kind;
    int unit;              // the segment's,
    int slice, last;       // and its slices: from, to

    // Before the first segment.
    __device__ __forceinline__ Segments(int from, int to)
        : end(to), warp(threadIdx.x >> 5), base(from), next(from), pair(-1), left(0), kind(kWhole), unit(0), slice(0), last(0) {}
    // Where the share of warp w starts among the slices of the round's units.
    __device__ __forceinline__ int share(const ExpertsSide& side, int w) const { return left * side.slices * w / kWarps; }
    __device__ __forceinline__ bool advance(const ExpertsSide& side) {
        const int tiles = side.tiles, slices = side.slices;
        if (kind == kGoOn) {   // the same round
            kind = kBegin;
            const int from = share(side, warp), to = share(side, warp + 1), u = divide(from + slices - 1, side.by_slices);
            unit = base + u;
            slice = 0;
            last = max(to - u * slices, 0);
            return true;
        }
        if (next >= end) return false;
        base = next;
        pair = divide(base, side.by_tiles);
        left = min(end, (pair + 1) * tiles) - base;
        if (left >= kWarps) {
            kind = kWhole;
            left = kWarps;
            unit = base + warp;
            slice = 0;
            last = slices;
        } else {
            kind = kGoOn;
            const int from = share(side, warp), to = share(side, warp + 1), u = divide(from, side.by_slices);
            unit = base + u;
            slice = from - u * slices;
            last = slice == 0 ? 0 : min(slices, slice + to - from);
        }
        next = base + left;
        return true;
    }
};

// A warp's slices on their way to shared memory, in the order in which it takes them: the codes as boxes of a tensor copy, whose
// 64-byte swizzle turns a row's four 16-byte pieces by (row / 2) % 4, the scales as a word for each lane's row; a barrier for each
// stage counts both.  (All of it by 16-byte asynchronous copies from the lanes: 15 clocks of the load pipe for 512 bytes, 2.6 us
// for the first four slices of 16 warps, and 101 us for 32 tokens where this took 93.)
template <int kStages>
struct Stream {
    const ExpertsSide& side;
    Pairs list;
    uint32_t codes, words, full;   // the warp's stages and their barriers
    int stage;                     // the next one to be filled
    Segments r;
    bool more;
    int first;                     // of the unit: its first row of all experts'
    const uint8_t* s;              // this lane's row's scales,
    int bytes;                     // to copy of them: none where there is no row

    __device__ __forceinline__ Stream(const ExpertsSide& sides, const Pairs& l, uint32_t c, uint32_t w, uint32_t f, int next, const Segments& segments)
        : side(sides), list(l), codes(c), words(w), full(f), stage(next), r(segments) {
        advance();
    }
    // To the next segment with slices.
    __device__ __forceinline__ void advance() {
        do more = r.advance(side);
        while (more && r.slice >= r.last);
        if (!more) return;
        const int e = static_cast<int>(list[r.pair] & 0xFFFFu);
        const int tile = r.unit - r.pair * side.tiles;
        first = e * side.rows + side.step * tile;
        const int lane = static_cast<int>(lane_id()), row = side.step * tile + (lane & 15) + (lane < 16 ? 0 : side.apart);
        const bool there = row < (lane < 16 ? side.half : side.rows);
        bytes = there ? 4 : 0;
        s = side.scales;
        if (there) {
            const int64_t group = static_cast<int64_t>(e) * ((side.rows + 127) / 128) + row / 128;
            s += (group * side.slices + r.slice) * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4;
        }
    }
    // Asks for the next slice, if there is one.
    __device__ __forceinline__ void ask() {
        if (!more) return;
        const uint32_t bar = full + 8 * stage;
        copy4(words + stage * kWordBytes + 4 * lane_id(), s, bytes);
        copies_arrive(bar);
        s += 512;
        if (lane_id() == 0) {
            mbar_arrive_expect_tx(bar, kSliceBytes);
            // what lies behind the end of either half is of no use, and does no harm
            const uint32_t to = codes + stage * kSliceBytes;
            tma_load_2d(to, &side.map, r.slice * (kSlice / 2), first, bar);
            tma_load_2d(to + kSliceBytes / 2, &side.map, r.slice * (kSlice / 2), first + side.apart, bar);
        }
        if (++stage == kStages) stage = 0;
        if (++r.slice == r.last) advance();
    }
};

// The unit's sums so far += one slice.  All places in shared memory; acts: this lane's place in the activations (row g, 16 bytes t of the slice's first
// block), `low` bytes further their low parts.
template <int kCols, bool kPairs, int kMost>
__device__ __forceinline__ void multiply(uint8_t* shared, int stage_codes, int stage_words, int scales, int acts, int pitch, int low,
                                         float (*acc)[kMost][4]) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2;
    // each lane turns one row's four bytes into factors, for all (48 instructions less than each for itself)
    const uint32_t w = *reinterpret_cast<const uint32_t*>(shared + stage_words + 4 * lane);
    *reinterpret_cast<uint4*>(shared + scales + 16 * lane) = make_uint4(scale_of(w, 0), scale_of(w, 1), scale_of(w, 2), scale_of(w, 3));
    __syncwarp();
    float by[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 f = *reinterpret_cast<const float4*>(shared + scales + 16 * (16 * m + 8 * h + g));
            by[m][h][0] = f.x;
            by[m][h][1] = f.y;
            by[m][h][2] = f.z;
            by[m][h][3] = f.w;
        }
    // the block's words of rows g, g + 8, g + 16 and g + 24 of the unit: this lane's is the address of its row, lane, at the block
    const uint32_t codes = smem_addr(shared + stage_codes + 64 * lane);
    const uint32_t turn = static_cast<uint32_t>((lane >> 1) & 3) << 4;
#pragma unroll
    for (int b = 0; b < kSlice / 32; ++b) {
        uint4 x[kCols], xl[kCols];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
            x[n] = *reinterpret_cast<const uint4*>(shared + acts + 8 * n * pitch + b * 64);
            if (kPairs) xl[n] = *reinterpret_cast<const uint4*>(shared + acts + low + 8 * n * pitch + b * 64);
        }
        uint32_t word[4];
        load_words4(word, codes + ((b << 4) ^ turn));
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            decode8(word[2 * m], lo);
            decode8(word[2 * m + 1], hi);
            const float s0 = by[m][0][b], s1 = by[m][1][b];
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
                float p[4];
                mma_first(p, lo[0], hi[0], lo[1], hi[1], x[n].x, x[n].y);
                mma(p, lo[2], hi[2], lo[3], hi[3], x[n].z, x[n].w);
                if (kPairs) {
                    mma(p, lo[0], hi[0], lo[1], hi[1], xl[n].x, xl[n].y);
                    mma(p, lo[2], hi[2], lo[3], hi[3], xl[n].z, xl[n].w);
                }
                acc[m][n][0] = fmaf(s0, p[0], acc[m][n][0]);
                acc[m][n][1] = fmaf(s0, p[1], acc[m][n][1]);
                acc[m][n][2] = fmaf(s1, p[2], acc[m][n][2]);
                acc[m][n][3] = fmaf(s1, p[3], acc[m][n][3]);
            }
        }
    }
}

// The rows of a pass, and their activations: x's lowered rows as they are, the rows of h as two fp16.
__device__ __forceinline__ void stage_rows(const ExpertsArgs& a, const ExpertsSide& side, Head* head, uint8_t* acts, const unsigned long long* masks,
                                           const float* weights, const float* backs, const uint16_t* ids, uint32_t pair) {
    const int e = static_cast<int>(pair & 0xFFFFu), skip = static_cast<int>(pair >> 16) * a.passes_rows;
    const int pitch = side.pitch, groups = side.groups;
    const unsigned long long mask = masks[e];
    const int rows = min(a.passes_rows, __popcll(mask) - skip);
    const bool here = !side.down && a.tokens <= kFew;
    __syncthreads();   // the rows before are done with
    if (threadIdx.x < kMaxPass) {
        Row row{-1, 0.0f, 0.0f, 0u};
        // a few tokens are their own columns of the first product, whatever they chose
        if (here ? (mask >> threadIdx.x & 1) != 0 : static_cast<int>(threadIdx.x) < rows) {
            unsigned long long m = mask;
#pragma unroll 1
            for (int i = here ? 0 : skip + static_cast<int>(threadIdx.x); i > 0; --i) m &= m - 1;
            const int token = here ? static_cast<int>(threadIdx.x) : __ffsll(static_cast<long long>(m)) - 1;
#pragma unroll 1
            for (int j = 0; j < a.top_k; ++j)   // an expert is among a token's choices once
                if (ids[token * a.top_k + j] == e) row.slot = token * a.top_k + j;
            row.weight = weights[row.slot];
            row.from = static_cast<uint32_t>(side.down ? row.slot : token);
            row.back = backs[row.from];
        }
        head->rows[threadIdx.x] = row;
        if (threadIdx.x == 0) {
            head->wide = rows > 8;
            head->slim = rows <= 4;
        }
    }
    __syncthreads();
    if (here) return;   // the activations are there
    if (!side.down) {
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * groups; i += kThreads) {
            const int n = divide(i, side.by_groups), c = i - n * groups;
            copy16(smem_addr(acts + n * pitch + 16 * c), a.lowered + (static_cast<int64_t>(head->rows[n].from) * groups + c) * 8, 16);
        }
        copies_commit();
        copies_wait<0>();
    } else {
        const bool wide = a.inner % 8 == 0;
#pragma unroll 2
        for (int i = threadIdx.x; i < rows * groups; i += kThreads) {
            const int n = divide(i, side.by_groups), c = 8 * (i - n * groups);
            const float* const p = a.h + static_cast<int64_t>(head->rows[n].from) * a.inner + c;
            float f[8];
            if (wide) {
                const bool in = c < a.inner;
                const float4 none = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const float4 u = in ? __ldcg(reinterpret_cast<const float4*>(p)) : none, v = in ? __ldcg(reinterpret_cast<const float4*>(p) + 1) : none;
                f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
                f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = c + j < a.inner ? __ldcg(p + j) : 0.0f;
            }
            const float up = 1.0f / head->rows[n].back;   // powers of two
            uint32_t w[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f[2 * j] * up, y = f[2 * j + 1] * up;
                w[j] = half2_of(x, y);
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                const float inf = __int_as_float(0x7F800000);
                l[j] = half2_of(fabsf(h.x) < inf ? x - h.x : 0.0f, fabsf(h.y) < inf ? y - h.y : 0.0f);
            }
            uint4* const to = reinterpret_cast<uint4*>(acts + n * pitch + 2 * c);
            *to = make_uint4(w[0], w[1], w[2], w[3]);
            to[(rows <= 4 ? 4 : a.passes_rows) * pitch / 16] = make_uint4(l[0], l[1], l[2], l[3]);
        }
    }
    __syncthreads();
}

// What becomes of a unit's sums, in the registers of one warp: element (row 16 m + 8 h + g, column 8 n + 2 t + c) of the
// unit in acc[m][n][2 h + c].
template <int kMost>
__device__ __forceinline__ void finish_up(const ExpertsArgs& a, const Head* head, int tile, int cols, const float (*acc)[kMost][4]) {
    const int g = static_cast<int>(lane_id()) >> 2, t = static_cast<int>(lane_id()) & 3;
#pragma unroll
    for (int n = 0; n < kMost; ++n) {
        if (n >= cols) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const Row row = head->rows[8 * n + 2 * t + c];
            float top = 0.0f;
            if (row.slot >= 0)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 16 * tile + 8 * h + g;
                    const float x = acc[0][n][2 * h + c] * row.back, u = acc[1][n][2 * h + c] * row.back;
                    const float v = x / (1.0f + expf(-x)) * u;
                    if (r < a.inner) {
                        a.h[static_cast<int64_t>(row.slot) * a.inner + r] = v;
                        top = fmaxf(top, finite_or_zero(v));
                    }
                }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            if (g == 0 && row.slot >= 0) atomicMax(a.tops + row.slot, __float_as_uint(top));   // the order does not matter
        }
    }
}

template <int kMost>
__device__ __forceinline__ void finish_down(const ExpertsArgs& a, const Head* head, int tile, int cols, const float (*acc)[kMost][4]) {
    const int g = static_cast<int>(lane_id()) >> 2, t = static_cast<int>(lane_id()) & 3;
#pragma unroll
    for (int n = 0; n < kMost; ++n) {
        if (n >= cols) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const Row row = head->rows[8 * n + 2 * t + c];
            if (row.slot < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 32 * tile + 8 * i + g;
                if (r < a.dim) a.part[static_cast<int64_t>(row.slot) * a.dim + r] = acc[i >> 1][n][2 * (i & 1) + c] * row.back * row.weight;
            }
        }
    }
}

// Phase 4: y from the experts' rows, in the order of the tokens' choices.
__device__ __forceinline__ void join(const ExpertsArgs& a, const float* weights) {
    const int all = a.tokens * a.dim;
#pragma unroll 1
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < all; i += gridDim.x * kThreads) {
        const int t = i / a.dim, r = i - t * a.dim;
        const float* const p = a.part + static_cast<int64_t>(t) * a.top_k * a.dim + r;
        const float* const w = weights + t * a.top_k;
        float sum = 0.0f;
#pragma unroll 1
        for (int j = 0; j < a.top_k; j += 8) {
            float v[8];   // all under way together; what no warp has left is not read
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = j + q < a.top_k && w[j + q] != 0.0f ? __ldcg(p + static_cast<int64_t>(j + q) * a.dim) : 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) sum += v[q];
        }
        const __nv_bfloat16 h = __float2bfloat16_rn(sum);
        a.y[t * a.ldy + r] = *reinterpret_cast<const uint16_t*>(&h);
    }
}

// A warp's stages.
struct Stages {
    int codes, words;     // their places in shared memory
    uint32_t full;        // their barriers
    int next;             // the stage that is taken next, and the parity of its barrier's phase
    uint32_t phase;
};

// A product over the CTA's range.
template <int kStages, int kMost>
__device__ __forceinline__ void product(const ExpertsArgs& a, const ExpertsSide& side, const Layout& at, uint8_t* shared, Segments seg,
                                        Stream<kStages>& stream, const Pairs& pairs, Stages& st) {
    Head* const head = reinterpret_cast<Head*>(shared);
    const int warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
    const int scales = at.scales + warp * kUnitRows * 16;
    const int pitch = side.pitch, low = a.passes_rows * pitch;
    float* const sums = reinterpret_cast<float*>(shared + at.sums) + lane;   // 32 lanes' values side by side, warp by warp
    constexpr int kValues = 8 * kMost;
    int pair = -1;
#pragma unroll 1
    while (seg.advance(side)) {
        if (seg.pair != pair) {
            pair = seg.pair;
            stage_rows(a, side, head, shared + at.acts, reinterpret_cast<const unsigned long long*>(shared + at.masks),
                                reinterpret_cast<const float*>(shared + at.weights), reinterpret_cast<const float*>(shared + at.backs),
                                reinterpret_cast<const uint16_t*>(shared + at.ids), pairs[pair]);
        }
        const bool down = side.down != 0, wide = kMost > 1 && head->wide != 0, slim = down && head->slim != 0;
        float acc[2][kMost][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kMost; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
        int x = at.acts + g * pitch + t * 16 + seg.slice * (kSlice * 2);
#pragma unroll 1
        for (int i = seg.slice; i < seg.last; ++i) {
            if (!mbar_wait(st.full + 8 * st.next, st.phase, a.err, kErrExperts, &head->abort)) {
                // No copies over copies, in this product or the next.  (A lane that gives up alone, for others ran out, leaves the
                // stage's next phase without its arrival: the others give up there.)
                stream.more = false;
                if (lane == 0 && head->lost[warp] == 0) head->lost[warp] = 1 + 2 * st.next + 256 * static_cast<int>(st.phase);
            }
            const int codes = st.codes + st.next * kSliceBytes, words = st.words + st.next * kWordBytes;
            if (kMost > 1 && wide) {
                if (down) multiply<kMost, true>(shared, codes, words, scales, x, pitch, low, acc);
                else multiply<kMost, false>(shared, codes, words, scales, x, pitch, low, acc);
            } else if (down && !slim) {
                multiply<1, true>(shared, codes, words, scales, x, pitch, low, acc);
            } else {
                multiply<1, false>(shared, codes, words, scales, x, pitch, low, acc);
            }
            __syncwarp();
            stream.ask();
            x += kSlice * 2;
            if (++st.next == kStages) {
                st.next = 0;
                st.phase ^= 1u;
            }
        }
        const int cols = wide ? kMost : 1;
        if (seg.kind == Segments::kGoOn) {   // the sums of a unit that another warp began, for that warp
            if (seg.slice < seg.last)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < kMost; ++n)
                        if (n < cols)
#pragma unroll
                            for (int i = 0; i < 4; ++i) sums[(warp * kValues + (n * 2 + m) * 4 + i) * 32] = acc[m][n][i];
            continue;
        }
        if (seg.kind == Segments::kBegin) {
            __syncthreads();   // the next write to the sums is behind a barrier of stage_rows or of the grid
            const int behind = (seg.unit - seg.base + 1) * side.slices;
            if (seg.last == 0) continue;
#pragma unroll 1
            for (int w = warp + 1; w < kWarps && seg.share(side, w) < behind; ++w) {
                if (seg.share(side, w) == seg.share(side, w + 1)) continue;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < kMost; ++n)
                        if (n < cols)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[m][n][i] += sums[(w * kValues + (n * 2 + m) * 4 + i) * 32];
            }
        }
        if (slim)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][0][i] += __shfl_xor_sync(0xFFFFFFFFu, acc[m][0][i], 2);   // columns 4 away
        const int tile = seg.unit - seg.pair * side.tiles;
        if (down) finish_down<kMost>(a, head, tile, cols, acc);
        else finish_up<kMost>(a, head, tile, cols, acc);
    }
}

// kMost: 8 kMost rows in a pass at most.
template <int kStages, int kMost>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ ExpertsArgs a) {
    extern __shared__ __align__(1024) uint8_t shared[];   // the swizzle goes by addresses
    const Layout at(a.experts, a.tokens, a.top_k, a.dim, a.inner, a.passes_rows, kStages);
    Head* const head = reinterpret_cast<Head*>(shared);
    float* const weights = reinterpret_cast<float*>(shared + at.weights);
    float* const backs = reinterpret_cast<float*>(shared + at.backs);
    uint16_t* const ids = reinterpret_cast<uint16_t*>(shared + at.ids);
    unsigned long long* const masks = reinterpret_cast<unsigned long long*>(shared + at.masks);
    uint32_t* const list = reinterpret_cast<uint32_t*>(shared + at.list);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        head->abort = 0;
        for (int w = 0; w < kWarps; ++w) head->lost[w] = 0;
        prefetch_tensormap(&a.side[0].map);
        prefetch_tensormap(&a.side[1].map);
    }
    if (threadIdx.x < kWarps * kStages)   // 32 lanes' words, and the codes
        mbar_init(smem_addr(&head->full[threadIdx.x / kStages][threadIdx.x % kStages]), 33);
    fence_barrier_init();

#pragma unroll 1
    for (int e = threadIdx.x; e < a.experts; e += kThreads) masks[e] = 0ull;
    if (threadIdx.x < kFew) head->tops[threadIdx.x] = 0u;
    __syncthreads();
    if (a.tokens <= kFew) {
        const int each = (kWarps - a.tokens) / a.tokens, mine = warp - a.tokens;   // warps of a row
        if (mine < 0) {
            choose(a, warp, weights, ids);
        } else if (mine < each * a.tokens) {
            const int t = mine / each;
            lower_row(a, t, 32 * (mine - t * each) + static_cast<int>(lane_id()), 32 * each, &head->tops[t], 32 * each * a.tokens,
                      reinterpret_cast<uint4*>(shared + at.acts + t * Layout::pitch(a.dim)), backs + t);
        }
        __syncthreads();
    } else {
#pragma unroll 1
        for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
            if (warp > 0)
                lower_row(a, t, static_cast<int>(threadIdx.x) - 32, kThreads - 32, &head->tops[0], kThreads - 32,
                          reinterpret_cast<uint4*>(a.lowered + static_cast<int64_t>(t) * ((Layout::pitch(a.dim) - 64) / 2)), a.backs + t);
            else choose(a, t, a.weights, a.ids);
            __syncthreads();
            if (threadIdx.x == 0) head->tops[0] = 0u;   // the next one's
            __syncthreads();
        }
        meet(a, 0);
    }
    list_pairs(a, head, masks, weights, ids, list, at.list_size, backs);
    const Pairs pairs{list, at.list_size, head->narrow};
    Stages st{at.codes + warp * kStages * kSliceBytes, at.words + warp * kStages * kWordBytes, smem_addr(head->full[warp]), 0, 0u};
    const uint32_t codes = smem_addr(shared + st.codes), words = smem_addr(shared + st.words);
#pragma unroll 1
    for (int p = 0; p < 2; ++p) {
        const ExpertsSide& side = a.side[p];
        const Segments seg(head->range[2 * p], head->range[2 * p + 1]);
        Stream<kStages> stream(side, pairs, codes, words, st.full, st.next, seg);
        __syncwarp();
        if (*static_cast<volatile int*>(&head->lost[warp]) != 0) stream.more = false;
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) stream.ask();
        if (p != 0) {
            meet(a, 1);
#pragma unroll 1
            for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads)   // a barrier of stage_rows is ahead of their use
                lift(__uint_as_float(__ldcg(a.tops + i)), backs + i);
        }
        product<kStages, kMost>(a, side, at, shared, seg, stream, pairs, st);
    }
    if (head->lost[warp] != 0 && lane_id() == 0) {   // copies from there on, which no wait has seen, may be on their way
        st.next = (head->lost[warp] & 255) / 2;
        st.phase = static_cast<uint32_t>(head->lost[warp] / 256);
        for (int i = 0; i < kStages; ++i) {
            mbar_wait_quiet(st.full + 8 * st.next, st.phase, kWaitLimitNs / 16);
            if (++st.next == kStages) st.next = 0, st.phase ^= 1u;
        }
    }
    meet(a, 2);
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < a.tokens * a.top_k; i += kThreads) a.tops[i] = 0u;   // for the next call
    join(a, weights);
    if (threadIdx.x == 0 && atomicAdd(&a.sync->left, 1u) == gridDim.x - 1u) {   // nobody looks at them any more
        a.sync->arrived[0] = a.sync->arrived[1] = a.sync->arrived[2] = 0u;
        a.sync->left = 0u;
    }
}

// Sets the rows of a pass and the stages, and gives the shared memory, or 0 where it does not fit.
int shape(ExpertsArgs* a) {
    // 16 rows where an expert has 8 on average, else 8: an expert with more than 8 is read twice then, but the others' stages
    // have the room (32 tokens, 8 of 64, 2048 x 1408: 93 us with 16, 85 with 8; 64 tokens, 2 of 8, 4096 x 2048: 74.5 and 77).
    for (int cols = a->tokens > 8 && a->tokens * a->top_k >= 8 * a->experts ? 2 : 1; cols >= 1; --cols) {
        a->passes_rows = 8 * cols;
        for (a->stages = 4; a->stages >= 2; --a->stages) {
            const Layout l(a->experts, a->tokens, a->top_k, a->dim, a->inner, a->passes_rows, a->stages);
            if (l.total <= kSharedMost) return l.total;
        }
    }
    return 0;
}

cudaError_t launch(ExpertsArgs a, int sms, cudaStream_t stream) {
    const auto by = [](int32_t d) { return d == 1 ? 0u : static_cast<uint32_t>(((uint64_t{1} << 32) + d - 1) / d); };
    for (ExpertsSide& s : a.side) {
        const uint64_t bytes = static_cast<uint64_t>(s.slices) * (kSlice / 2);
        s.pitch = Layout::pitch(s.k);
        s.groups = s.slices * (kSlice / 8);
        s.by_tiles = by(s.tiles);
        s.by_slices = by(s.slices);
        s.by_groups = by(s.groups);
        if (!encode_map_2d(&s.map, CU_TENSOR_MAP_DATA_TYPE_UINT8, s.codes, bytes, static_cast<uint64_t>(s.rows) * a.experts, bytes, kSlice / 2,
                           kUnitRows / 2, CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    using K = void (*)(ExpertsArgs);
    static const K kernels[2][3] = {{experts_kernel<2, 1>, experts_kernel<3, 1>, experts_kernel<4, 1>},
                                    {experts_kernel<2, 2>, experts_kernel<3, 2>, experts_kernel<4, 2>}};
    const int smem = shape(&a);
    if (smem == 0) return cudaErrorInvalidValue;
    const K kernel = kernels[a.passes_rows > 8][a.stages - 2];
    static std::atomic<uint64_t> known[2][3];   // the devices that have the attribute: the call costs the host as much as a launch
    std::atomic<uint64_t>& devices = known[a.passes_rows > 8][a.stages - 2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(devices.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedMost);
        if (e != cudaSuccess) return e;
        devices.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int64_t align256(int64_t n) { return (n + 255) & ~int64_t{255}; }

// Sizes that the kernel takes: what it needs of shared memory decides.
bool sizes_ok(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t inner) {
    if (tokens < 0 || tokens > MXFP4_EXPERTS_MAX_TOKENS || experts < 1 || experts > MXFP4_MAX_GROUPS || top_k < 1 ||
        top_k > MXFP4_EXPERTS_MAX_TOP_K || top_k > experts || dim < 1 || dim > 65536 || inner < 1 || inner > 65536)
        return false;
    ExpertsArgs a = {};
    a.experts = static_cast<int32_t>(experts);
    a.tokens = static_cast<int32_t>(tokens > 0 ? tokens : 1);
    a.top_k = static_cast<int32_t>(top_k);
    a.dim = static_cast<int32_t>(dim);
    a.inner = static_cast<int32_t>(inner);
    return shape(&a) != 0;
}

// The workspace: parts at multiples of 256 bytes.
struct Parts {
    int64_t weights, ids, tops, backs, lowered, h, part, total;
    Parts(int64_t tokens, int64_t top_k, int64_t dim, int64_t inner) {
        const int64_t choices = tokens * top_k;
        tops = align256(sizeof(ExpertsSync));   // at the same place in every call: each leaves them zero
        weights = tops + 4 * MXFP4_EXPERTS_MAX_TOKENS * MXFP4_EXPERTS_MAX_TOP_K;
        ids = weights + align256(4 * choices);
        backs = ids + align256(2 * choices);
        lowered = backs + align256(4 * tokens);
        h = lowered + align256(2 * tokens * ((dim + kSlice - 1) / kSlice * kSlice));
        part = h + align256(4 * choices * inner);
        total = part + align256(4 * choices * dim);
    }
};

}  // namespace
}  // namespace mxfp4

extern "C" {

mxfp4_status mxfp4_experts_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t inner, size_t* bytes) {
    if (!mxfp4::sizes_ok(tokens, experts, top_k, dim, inner) || bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(mxfp4::Parts(tokens, top_k, dim, inner).total);
    return MXFP4_OK;
}

mxfp4_status mxfp4_experts_forward(const void* x, int64_t tokens, int64_t ldx, const void* logits, int64_t ldl, int64_t experts,
                                   int64_t top_k, int64_t dim, int64_t inner, const void* up_q, const void* up_s,
                                   const void* down_q, const void* down_s, void* y, int64_t ldy, int32_t flags, void* workspace,
                                   size_t workspace_bytes, mxfp4_stream_t stream) {
    size_t need = 0;
    if (mxfp4_experts_workspace_bytes(tokens, experts, top_k, dim, inner, &need) != MXFP4_OK || (flags & ~3))
        return MXFP4_ERR_INVALID_ARG;
    const int64_t most = int64_t{1} << 40;
    if (tokens > 0 && (!x || !logits || !up_q || !up_s || !down_q || !down_s || !y || !workspace || workspace_bytes < need ||
                       (tokens > 1 && (ldx < dim || ldl < experts || ldy < dim || ldx > most || ldl > most || ldy > most))))
        return MXFP4_ERR_INVALID_ARG;
    if (!mxfp4::aligned_to(x, 2) || !mxfp4::aligned_to(y, 2) || !mxfp4::aligned_to(logits, flags & MXFP4_EXPERTS_LOGITS_F32 ? 4 : 2) ||
        !mxfp4::aligned_to(up_q, 16) || !mxfp4::aligned_to(up_s, 16) || !mxfp4::aligned_to(down_q, 16) ||
        !mxfp4::aligned_to(down_s, 16) || !mxfp4::aligned_to(workspace, 256))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK || tokens == 0) return static_cast<mxfp4_status>(st);
    mxfp4::ExpertsArgs a = {};
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = tokens > 1 ? ldx : 0;
    a.logits = logits;
    a.ldl = tokens > 1 ? ldl : 0;
    const mxfp4::Parts parts(tokens, top_k, dim, inner);
    a.sync = reinterpret_cast<mxfp4::ExpertsSync*>(w);
    a.weights = reinterpret_cast<float*>(w + parts.weights);
    a.ids = reinterpret_cast<uint16_t*>(w + parts.ids);
    a.tops = reinterpret_cast<uint32_t*>(w + parts.tops);
    a.backs = reinterpret_cast<float*>(w + parts.backs);
    a.lowered = reinterpret_cast<uint16_t*>(w + parts.lowered);
    a.h = reinterpret_cast<float*>(w + parts.h);
    a.part = reinterpret_cast<float*>(w + parts.part);
    a.err = err;
    a.y = static_cast<uint16_t*>(y);
    a.ldy = tokens > 1 ? ldy : 0;
    a.tokens = static_cast<int32_t>(tokens);
    a.experts = static_cast<int32_t>(experts);
    a.top_k = static_cast<int32_t>(top_k);
    a.dim = static_cast<int32_t>(dim);
    a.inner = static_cast<int32_t>(inner);
    a.logits_f32 = flags & MXFP4_EXPERTS_LOGITS_F32 ? 1 : 0;
    a.normalize = flags & MXFP4_EXPERTS_NORMALIZE ? 1 : 0;
    const int32_t d = a.dim, n = a.inner;
    const auto set = [&](mxfp4::ExpertsSide& s, const void* q, const void* scales, int32_t rows, int32_t k, int32_t step, int32_t apart, int32_t half) {
        s.codes = static_cast<const uint8_t*>(q);
        s.scales = static_cast<const uint8_t*>(scales);
        s.rows = rows;
        s.k = k;
        s.step = step;
        s.apart = apart;
        s.half = half;
        s.tiles = (half + step - 1) / step;
        s.slices = (k + mxfp4::kSlice - 1) / mxfp4::kSlice;
    };
    set(a.side[0], up_q, up_s, 2 * n, d, 16, n, n);
    set(a.side[1], down_q, down_s, d, n, 32, 16, d);
    a.side[1].down = 1;
    return mxfp4::launch(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

}  // extern "C"
