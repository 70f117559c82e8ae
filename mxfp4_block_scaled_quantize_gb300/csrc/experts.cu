// experts.cu -- a whole mixture-of-experts layer for a few tokens, in two kernels.
//
//   p = softmax(logits), the top_k largest of them (ties: the lowest index), w = p or p / sum of the chosen p,
//   y_t = sum over the chosen experts e of w_e W2_e . (silu(g) u),   [g; u] = W1_e . x_t,   silu(g) = g / (1 + exp(-g)),
//   W1 [E, 2 inner, dim], W2 [E, dim, inner] in MXFP4 (E2M1 codes, an E8M0 scale for 32 along the row).
//
// For a few tokens the time is that of the chosen experts' weights, each read once: 17 / 32 bytes an element at 23 bytes a
// clock and SM.  So the activations stay as they are (rounding them to 4 bits would save nothing), and a product has the
// weights as the 16 rows of a small matrix instruction (mma.sync m16n8k16: the tensor pipe is at a tenth of its rate here, and
// the tcgen05 forms would want 128 rows of one expert and 4-bit or 8-bit activations) and up to 16 routed rows
// as its columns.
//
// Numbers.  A code is exact in fp16.  x is bf16 times a power of two that brings its row's largest value to 2^14 .. 2^15: exact
// in fp16 but for what lies 2^-29 and more below that.  The activations between the products are fp32, and the second
// product takes them as the sum of two fp16 (22 bits).  A block of 32 is summed by the matrix instruction in fp32 and then
// multiplied by its scale in fp32, as all sums are.  y is rounded once.
//
// Work.  A unit is 32 rows of an expert's weights (16 of g and the same 16 of u) against a pass of its routed rows.  A CTA, one
// an SM, takes a range of consecutive units, so it stages an expert's activations in shared memory once.  Its 16 warps take
// 16 units of one expert at a time, a whole unit each, and meet nobody; of the n < 16 that are left they take 8, 4, 2 and 1, as n
// has them, with 2, 4, 8 and 16 warps to a unit, each with its part of the row's length: so all warps do the same whatever n is.
// (All units dealt out in slices of 128 elements to 16 warps, which met after each one: 171 instructions for 32 x 32 weights, and
// 255 us where it is now ##.)  Each warp has several slices (2 KB of codes) on their way to shared memory by asynchronous
// copies of its own, across the ends of its units.
//   Rows of a unit: 32 q + i for q = 0 .. 3 and a few consecutive i of a group of 128, so that their scales (16 bytes for the
//   four q of one i in the scale layout) are consecutive too.
//   The sum over experts: each unit of the second product leaves its rows, weighted, in fp32; the CTA that
//   leaves the last one for 32 columns adds them up in the order of the tokens' choices, when it is done with its units.  No CTA waits for another, and the
//   order of additions is fixed by the call's routing.
//
// The routing is so little work (64 tokens of 64 experts: 1 us) that every CTA does it for itself; the second kernel does
// it, and asks for its first weights, while the first one is still at work.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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
constexpr int kStageBytes = kSliceBytes + 4 * kUnitRows; // and a word of four scales for each row
constexpr int kMaxPass = 16;                             // routed rows of a pass
constexpr int kSharedMost = 227 * 1024;

struct Row {           // of a pass
    int32_t token;
    int32_t slot;      // token * top_k + place among the token's choices; -1: not routed here
    float back;        // undoes the power of two of its activations
    float weight;
};

// Shared memory: this head, then [experts] masks, [tokens * top_k] weights and experts, the list of (expert, pass),
// [tiles] the queue of finished tiles, the activations, the units' sums, the warps' scales and their stages.
struct Head {
    Row rows[kMaxPass];
    int32_t narrow;    // (expert, pass) pairs of up to 8 rows,
    int32_t pairs;     // and all of them
    int32_t wide;      // the pass has more than 8 rows
    int32_t queued;    // of the tiles whose last unit one of this CTA's warps left
    uint32_t top[kMaxPass];   // largest magnitudes of the pass's activations, as bits
};

__host__ __device__ inline int align16(int n) { return (n + 15) & ~15; }

struct Layout {
    int masks, weights, ids, list, list_size, queue, acts, sums, scales, stages, total;
    __host__ __device__ Layout(int experts, int tokens, int top_k, int k, int tiles, int pass_rows, bool pairs, int stage_count) {
        const int choices = tokens * top_k;
        masks = align16(sizeof(Head));
        weights = masks + align16(8 * experts);
        ids = weights + align16(4 * choices);
        list = ids + align16(2 * choices);
        // an expert's passes: one, and one more for every further pass_rows of its tokens
        list_size = (experts < choices ? experts : choices) + choices / pass_rows;
        queue = list + align16(4 * list_size);
        acts = queue + (pairs ? align16(2 * tiles) : 0);
        sums = acts + pass_rows * pitch(k) * (pairs ? 2 : 1);
        scales = sums + kWarps / 2 * kUnitRows * kMaxPass * 4;
        stages = scales + kWarps * kUnitRows * 16;
        total = stages + kWarps * stage_count * kStageBytes;
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

// The choices of kTokens tokens from t on (those below a.tokens).  kPer: 32 kPer experts at most.  Order: value, then lowest
// index; a NaN is above all values, as in a sort.  Several tokens' chains of warp-wide steps run beside each other.
template <int kPer, int kTokens>
__device__ __forceinline__ void choose(const ExpertsArgs& a, int t, unsigned long long* masks, float* weights, uint16_t* ids) {
    const int lane = static_cast<int>(lane_id());
    const float none = __int_as_float(0xFF800000);
    float v[kTokens][kPer];
    uint32_t key[kTokens][kPer];
#pragma unroll
    for (int x = 0; x < kTokens; ++x)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = i * 32 + lane;
            v[x][i] = e < a.experts && t + x < a.tokens ? logit_of(a, t + x, e) : 0.0f;
        }
#pragma unroll
    for (int x = 0; x < kTokens; ++x)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const uint32_t u = __float_as_uint(v[x][i] + 0.0f);   // one zero
            key[x][i] = v[x][i] != v[x][i] ? 0xFFFFFFFFu : u & 0x80000000u ? ~u : u | 0x80000000u;
            if (i * 32 + lane >= a.experts) key[x][i] = 0u;       // below every value
        }
    float mine[kTokens], top[kTokens];   // lane j: the value of choice j
    int id[kTokens];
#pragma unroll
    for (int x = 0; x < kTokens; ++x) mine[x] = top[x] = 0.0f, id[x] = 0;
#pragma unroll 1
    for (int j = 0; j < a.top_k; ++j)
#pragma unroll
        for (int x = 0; x < kTokens; ++x) {
            uint32_t best = 0u;
            int at = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (key[x][i] > best) {
                    best = key[x][i];
                    at = i;
                }
            const uint32_t most = max_all(best);
            const int e = static_cast<int>(min_all(best == most ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu));
            float value = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i * 32 + lane == e) {
                    key[x][i] = 0u;
                    value = v[x][i];
                }
            value = __shfl_sync(0xFFFFFFFFu, value, e & 31);
            if (j == 0) top[x] = value;
            if (lane == j) {
                mine[x] = value;
                id[x] = e;
            }
        }
#pragma unroll
    for (int x = 0; x < kTokens; ++x) {
        const float p = lane < a.top_k && mine[x] != none ? expf(mine[x] - top[x]) : 0.0f;
        float sum = p;
        if (!a.normalize) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i * 32 + lane < a.experts && v[x][i] != none) sum += expf(v[x][i] - top[x]);
        }
        sum = sum_all(sum);
        if (lane < a.top_k && t + x < a.tokens) {
            const float w = sum == 0.0f ? 0.0f : p / sum;   // 0: every logit is -inf
            weights[(t + x) * a.top_k + lane] = w;
            ids[(t + x) * a.top_k + lane] = static_cast<uint16_t>(id[x]);
            if (w != 0.0f) atomicOr(&masks[id[x]], 1ull << (t + x));   // not where it changes nothing
        }
    }
}

// The routing: each expert's tokens, and the list of (expert, pass) pairs that have any: those of up to 8 rows from its front
// on, the others from its back on.
__device__ void route(const ExpertsArgs& a, Head* head, unsigned long long* masks, float* weights, uint16_t* ids, uint32_t* list, int list_size) {
    for (int e = threadIdx.x; e < a.experts; e += kThreads) masks[e] = 0ull;
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (a.experts <= 64) {
        if (a.tokens <= kWarps) {
            if (warp < a.tokens) choose<2, 1>(a, warp, masks, weights, ids);
        } else {
#pragma unroll 1
            for (int t = 2 * warp; t < a.tokens; t += 2 * kWarps) choose<2, 2>(a, t, masks, weights, ids);
        }
    } else if (a.experts <= 256) {
#pragma unroll 1
        for (int t = warp; t < a.tokens; t += kWarps) choose<8, 1>(a, t, masks, weights, ids);
    } else {
#pragma unroll 1
        for (int t = warp; t < a.tokens; t += kWarps) choose<32, 1>(a, t, masks, weights, ids);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = static_cast<int>(lane_id());
        if (lane == 0) head->queued = 0;
        int before = 0;   // pairs of the experts before: narrow ones, and 2^16 times the wide ones
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            const int e = e0 + lane;
            const int n = e < a.experts ? __popcll(masks[e]) : 0;
            const int full = n / a.passes_rows, rest = n - full * a.passes_rows;
            const int wide = a.passes_rows > 8 ? full + (rest > 8) : 0;
            const int mine = (full + (rest > 0) - wide) | wide << 16;
            int sum = mine;   // inclusive over the lanes
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
                if (lane >= d) sum += up;
            }
            int at = before + sum - mine;
            for (int p = 0; p < full + (rest > 0); ++p) {
                const bool is_wide = p < wide;   // full passes first, the one with the rest last
                list[is_wide ? list_size - 1 - (at >> 16) : at & 0xFFFF] = static_cast<uint32_t>(e) | static_cast<uint32_t>(p) << 16;
                at += is_wide ? 1 << 16 : 1;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) {
            head->narrow = before & 0xFFFF;
            head->pairs = (before & 0xFFFF) + (before >> 16);
        }
    }
    __syncthreads();
}

// Pair p of the list, those of up to 8 rows first.
struct Pairs {
    const uint32_t* list;
    int size, narrow;
    __device__ __forceinline__ uint32_t operator[](int p) const { return list[p < narrow ? p : size - 1 - (p - narrow)]; }
};

// What each of the two kernels multiplies.
struct Up {
    static constexpr bool kPairs = false;
    // The weights' row for row lr of tile `tile`; -1: none.
    __device__ __forceinline__ static int row(const ExpertsArgs& a, int tile, int lr) {
        const int r = hidden(tile, lr & 15);
        return r < a.inner ? (lr < 16 ? r : a.inner + r) : -1;
    }
    __device__ __forceinline__ static int hidden(int tile, int m) {
        return 128 * (tile >> 3) + 32 * (m & 3) + 4 * (tile & 7) + (m >> 2);
    }
};
struct Down {
    static constexpr bool kPairs = true;
    __device__ __forceinline__ static int row(const ExpertsArgs& a, int tile, int lr) {
        const int m = lr & 15, r = 128 * (tile >> 2) + 32 * (m & 3) + 8 * (tile & 3) + 4 * (lr >> 4) + (m >> 2);
        return r < a.dim ? r : -1;
    }
};

// A warp's way through the CTA's units, round by round: 16 units of one expert and pass with a warp each, or the 8, 4, 2 or 1
// that are left with more warps to each.
struct Rounds {
    int end, tiles, slices, warp;
    int base;              // first unit of the round
    int next;              // and of the one after it
    int pair;              // the round's place in the list of (expert, pass)
    int parts;             // warps of a unit
    int unit, part;        // this warp's
    int slice, last;       // its slices: from, to

    // Before the first round.
    __device__ __forceinline__ Rounds(int from, int to, int tiles_, int slices_)
        : end(to), tiles(tiles_), slices(slices_), warp(threadIdx.x >> 5), base(from), next(from), pair(-1), parts(1), unit(0), part(0),
          slice(0), last(0) {}
    __device__ __forceinline__ bool advance() {
        if (next >= end) return false;
        base = next;
        pair = base / tiles;
        const int left = min(end, (pair + 1) * tiles) - base;
        const int shift = left >= kWarps ? 0 : __clz(left) - (31 - 4);   // kWarps = 2^4
        parts = 1 << shift;
        unit = base + (warp >> shift);
        part = warp & (parts - 1);
        slice = (slices * part) >> shift;
        last = (slices * (part + 1)) >> shift;
        next = base + (kWarps >> shift);
        return true;
    }
};

// A warp's slices on their way to shared memory, in the order in which it takes them.
template <typename Product, int kStages>
struct Stream {
    const ExpertsArgs& a;
    Pairs list;
    uint32_t to, end_to, d;   // the warp's stages, and the next one to be filled
    Rounds r;
    bool more;
    const uint8_t* q[4];      // this lane's piece of four rows
    const uint8_t* s;         // and its row's scales
    int bytes[5];             // to copy of each: none where there is no row

    __device__ __forceinline__ Stream(const ExpertsArgs& args, const Pairs& l, uint32_t stages, const Rounds& rounds)
        : a(args), list(l), to(stages), end_to(stages + kStages * kStageBytes), d(stages), r(rounds) {
        advance();
    }
    // To the next round with slices for this warp.
    __device__ __forceinline__ void advance() {
        do more = r.advance();
        while (more && r.slice >= r.last);
        if (!more) return;
        const int tile = r.unit - r.pair * a.tiles, lane = static_cast<int>(lane_id());
        const int64_t e = list[r.pair] & 0xFFFFu;
        const int64_t pitch = static_cast<int64_t>(r.slices) * (kSlice / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = Product::row(a, tile, 8 * i + (lane >> 2));
            bytes[i] = row < 0 ? 0 : 16;
            q[i] = a.q + (row < 0 ? 0 : (e * a.rows + row) * pitch + r.slice * (kSlice / 2) + (lane & 3) * 16);
        }
        const int row = Product::row(a, tile, lane);
        const int64_t atom = (e * ((a.rows + 127) / 128) + row / 128) * r.slices + r.slice;
        bytes[4] = row < 0 ? 0 : 4;
        s = a.s + (row < 0 ? 0 : atom * 512 + (row & 31) * 16 + ((row & 127) >> 5) * 4);
    }
    // Asks for the next slice, or for nothing: a group of copies either way.
    __device__ __forceinline__ void ask() {
        if (more) {
            const int lane = static_cast<int>(lane_id());
            // row 8 i + lane / 4 at 64 bytes of it, its 16-byte pieces turned by (row / 2) % 4
            const uint32_t at = d + static_cast<uint32_t>((lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                copy16(at + 512 * i, q[i], bytes[i]);
                q[i] += kSlice / 2;
            }
            copy4(d + static_cast<uint32_t>(kSliceBytes + 4 * lane), s, bytes[4]);
            s += 512;
            d += kStageBytes;
            if (d == end_to) d = to;
            if (++r.slice == r.last) advance();
        }
        copies_commit();
    }
};

// The unit's sums so far += one slice.  acts: this lane's place in the activations (row g, 16 bytes t of the slice's first
// block), `low` bytes further their low parts.
template <int kCols, bool kPairs, int kMost>
__device__ __forceinline__ void multiply(const uint8_t* stage, float4* scales, const uint8_t* acts, int pitch, int low,
                                         float (*acc)[kMost][4]) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
    // each lane turns one row's four bytes into factors, for all (48 instructions less than each for itself)
    const uint32_t w = reinterpret_cast<const uint32_t*>(stage + kSliceBytes)[lane];
    reinterpret_cast<uint4*>(scales)[lane] = make_uint4(scale_of(w, 0), scale_of(w, 1), scale_of(w, 2), scale_of(w, 3));
    __syncwarp();
    float by[2][2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 f = scales[16 * m + 8 * h + g];
            by[m][h][0] = f.x;
            by[m][h][1] = f.y;
            by[m][h][2] = f.z;
            by[m][h][3] = f.w;
        }
    const uint8_t* const codes = stage + g * 64 + t * 4;
    const int turn = ((g >> 1) & 3) << 4;
#pragma unroll
    for (int b = 0; b < kSlice / 32; ++b) {
        uint4 x[kCols], xl[kCols];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
            x[n] = *reinterpret_cast<const uint4*>(acts + 8 * n * pitch + b * 64);
            if (kPairs) xl[n] = *reinterpret_cast<const uint4*>(acts + low + 8 * n * pitch + b * 64);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t lo[4], hi[4];
            decode8(*reinterpret_cast<const uint32_t*>(codes + 1024 * m + ((b << 4) ^ turn)), lo);
            decode8(*reinterpret_cast<const uint32_t*>(codes + 1024 * m + 512 + ((b << 4) ^ turn)), hi);
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

__device__ __forceinline__ float x_of(const ExpertsArgs& a, int64_t row, int c) {
    return c < a.k ? __uint_as_float(static_cast<uint32_t>(__ldg(a.x + row * a.ldx + c)) << 16) : 0.0f;
}

// Eight elements of x's row from c on.
__device__ __forceinline__ void x8(const ExpertsArgs& a, int64_t row, int c, bool wide, float* f) {
    if (wide && c < a.k) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(a.x + row * a.ldx + c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = x_of(a, row, c + i);
}

// Eight elements of the row of h from c on.
__device__ __forceinline__ void h8(const ExpertsArgs& a, int64_t row, int c, bool wide, float* f) {
    const float* const p = a.h + row * a.inner + c;
    if (wide && c < a.k) {
        const float4 u = __ldcg(reinterpret_cast<const float4*>(p)), v = __ldcg(reinterpret_cast<const float4*>(p) + 1);
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < a.k ? __ldcg(p + i) : 0.0f;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The rows of a pass and their activations.  `all`: the first product of few tokens, whose rows are all tokens
// whatever the expert: `staged` then says that they are there already.
template <typename Product>
__device__ void stage_rows(const ExpertsArgs& a, Head* head, uint8_t* acts, const unsigned long long* masks, const float* weights,
                           const uint16_t* ids, uint32_t pair, bool all, bool staged) {
    const int e = static_cast<int>(pair & 0xFFFFu), pass = static_cast<int>(pair >> 16);
    const int pitch = Layout::pitch(a.k), rows = a.passes_rows;
    __syncthreads();   // the rows before are done with
    if (threadIdx.x < static_cast<unsigned>(rows)) {
        const int n = threadIdx.x;
        unsigned long long m = masks[e];
        int token = -1, slot = -1;
        if (all) {
            token = n < a.tokens ? n : -1;
        } else {
            int skip = pass * rows + n;
            for (; skip > 0 && m != 0; --skip) m &= m - 1;
            token = m != 0 ? __ffsll(static_cast<long long>(m)) - 1 : -1;
        }
        if (token >= 0 && (masks[e] >> token & 1ull))
            for (int j = 0; j < a.top_k; ++j)   // an expert is among a token's choices once
                if (ids[token * a.top_k + j] == e) slot = token * a.top_k + j;
        head->rows[n].token = token;
        head->rows[n].slot = slot;
        head->rows[n].weight = slot >= 0 ? weights[slot] : 0.0f;
        if (!staged) head->top[n] = 0u;
        if (n == rows - 1) head->wide = rows > 8 && (all ? a.tokens : __popcll(masks[e]) - pass * rows) > 8;
    }
    __syncthreads();
    if (!staged) {
        // All threads over the rows' groups of 8: the largest magnitudes (whose order does not matter), then the values, with up
        // to kHeld groups of a thread in registers in between; those beyond are read twice.
        constexpr int kHeld = Product::kPairs ? 2 : 4;
        const int groups = (pitch - 64) / 16;
        int last = rows;   // rows that there are: what the others' columns give is not used
        if (!all) last = min(rows, __popcll(masks[e]) - pass * rows);
        else last = a.tokens;
        const int all_groups = last * groups;
        auto load = [&](int i, float* f) {
            const int n = i / groups, c = 8 * (i - n * groups);
            const int64_t row = Product::kPairs ? head->rows[n].slot : head->rows[n].token;
            if (Product::kPairs) h8(a, row, c, a.inner % 8 == 0, f);
            else x8(a, row, c, a.k % 8 == 0 && (reinterpret_cast<uintptr_t>(a.x + row * a.ldx) & 15u) == 0, f);
        };
        auto largest = [&](int i, const float* f) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_or_zero(f[j]));
            uint32_t bits = __float_as_uint(top);
            if (groups % 32 == 0) {   // a warp's groups are of one row
                bits = max_all(bits);
                if (lane_id() != 0) return;
            }
            atomicMax(&head->top[i / groups], bits);
        };
        auto place = [&](int i, const float* f) {
            const int n = i / groups;
            float back;
            const float up = lift(__uint_as_float(head->top[n]), &back);
            uint32_t w[4], l[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = f[2 * j] * up, q = f[2 * j + 1] * up;
                w[j] = half2_of(p, q);
                if (Product::kPairs) {
                    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                    const float inf = __int_as_float(0x7F800000);
                    l[j] = half2_of(fabsf(h.x) < inf ? p - h.x : 0.0f, fabsf(h.y) < inf ? q - h.y : 0.0f);
                }
            }
            uint4* const to = reinterpret_cast<uint4*>(acts + n * pitch) + (i - n * groups);
            *to = make_uint4(w[0], w[1], w[2], w[3]);
            if (Product::kPairs) to[rows * pitch / 16] = make_uint4(l[0], l[1], l[2], l[3]);
        };
        float held[kHeld][8];
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (threadIdx.x + h * kThreads < all_groups) load(threadIdx.x + h * kThreads, held[h]);
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (threadIdx.x + h * kThreads < all_groups) largest(threadIdx.x + h * kThreads, held[h]);
#pragma unroll 1
        for (int i = threadIdx.x + kHeld * kThreads; i < all_groups; i += kThreads) {
            float f[8];
            load(i, f);
            largest(i, f);
        }
        __syncthreads();
        if (threadIdx.x < static_cast<unsigned>(rows)) {
            float back;
            lift(__uint_as_float(head->top[threadIdx.x]), &back);
            head->rows[threadIdx.x].back = back;
        }
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
            if (threadIdx.x + h * kThreads < all_groups) place(threadIdx.x + h * kThreads, held[h]);
#pragma unroll 1
        for (int i = threadIdx.x + kHeld * kThreads; i < all_groups; i += kThreads) {
            float f[8];
            load(i, f);
            place(i, f);
        }
    }
    __syncthreads();
}

// What becomes of a unit's sums, in the registers of one warp: element (row 16 m + 8 h + g, column 8 n + 2 t + c) of the
// unit in acc[m][n][2 h + c].
template <int kMost>
__device__ __forceinline__ void finish(Up, const ExpertsArgs& a, Head* head, uint16_t*, int tile, int cols,
                                       const float (*acc)[kMost][4]) {
    const int g = static_cast<int>(lane_id()) >> 2, t = static_cast<int>(lane_id()) & 3;
#pragma unroll
    for (int n = 0; n < kMost; ++n) {
        if (n >= cols) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const Row row = head->rows[8 * n + 2 * t + c];
            if (row.slot < 0) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = Up::hidden(tile, 8 * h + g);
                const float x = acc[0][n][2 * h + c] * row.back, u = acc[1][n][2 * h + c] * row.back;
                if (r < a.inner) a.h[static_cast<int64_t>(row.slot) * a.inner + r] = x / (1.0f + expf(-x)) * u;
            }
        }
    }
}

template <int kMost>
__device__ __forceinline__ void finish(Down, const ExpertsArgs& a, Head* head, uint16_t* queue, int tile, int cols,
                                       const float (*acc)[kMost][4]) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < kMost; ++n) {
        if (n >= cols) break;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const Row row = head->rows[8 * n + 2 * t + c];
            if (row.slot < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = Down::row(a, tile, 8 * i + g);
                if (r >= 0) __stcg(a.part + static_cast<int64_t>(row.slot) * a.dim + r, acc[i >> 1][n][2 * (i & 1) + c] * row.back * row.weight);
            }
        }
    }
    __threadfence();
    __syncwarp();
    if (lane == 0 && atomicAdd(a.done + tile, 1u) == static_cast<uint32_t>(head->pairs) - 1u) {
        __threadfence();
        queue[atomicAdd(&head->queued, 1)] = static_cast<uint16_t>(tile);
    }
}

// The sums over the experts for the tiles in the queue: a warp for four of a tile's tokens, a lane for each of its columns.
__device__ __forceinline__ void join(const ExpertsArgs& a, const Head* head, const uint16_t* queue, const float* weights) {
    constexpr int kTogether = 4;
    const int lane = static_cast<int>(lane_id()), fours = (a.tokens + kTogether - 1) / kTogether;
#pragma unroll 1
    for (int i = threadIdx.x >> 5; i < head->queued * fours; i += kWarps) {
        const int tile = queue[i / fours], t = i % fours * kTogether, r = Down::row(a, tile, lane);
        if (t == 0 && lane == 0) a.done[tile] = 0u;
        if (r < 0) continue;
        const int choices = min(kTogether, a.tokens - t) * a.top_k;
        const float* const p = a.part + static_cast<int64_t>(t) * a.top_k * a.dim + r;
        const float* const w = weights + t * a.top_k;
        float sum[kTogether] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int j = 0; j < a.top_k; j += 4) {
            float v[4][kTogether];   // all under way together; what no warp has left is not read
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int x = 0; x < kTogether; ++x) {
                    const int c = x * a.top_k + j + q;
                    v[q][x] = j + q < a.top_k && c < choices && w[c] != 0.0f ? __ldcg(p + static_cast<int64_t>(c) * a.dim) : 0.0f;
                }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int x = 0; x < kTogether; ++x) sum[x] += v[q][x];
        }
#pragma unroll
        for (int x = 0; x < kTogether; ++x) {
            const __nv_bfloat16 h = __float2bfloat16_rn(sum[x]);
            if (t + x < a.tokens) a.y[(t + x) * a.ldy + r] = *reinterpret_cast<const uint16_t*>(&h);
        }
    }
}

// A wide unit takes 1.6 times as long as one of up to 8 rows.
constexpr uint32_t kNarrowCost = 5, kWideCost = 8;

// The unit at which CTA `cta` starts, so that all have the same to do.
__device__ __forceinline__ int range_start(const Head* head, int tiles, uint32_t cta) {
    const uint32_t narrow = static_cast<uint32_t>(head->narrow * tiles), all = static_cast<uint32_t>(head->pairs * tiles);
    // below 2^32: at most 2^11 pairs of 300 tiles on 152 SMs
    const uint32_t at = (narrow * kNarrowCost + (all - narrow) * kWideCost) * cta / gridDim.x;
    return static_cast<int>(at < narrow * kNarrowCost ? at / kNarrowCost : narrow + (at - narrow * kNarrowCost) / kWideCost);
}

// kMost: 8 kMost rows in a pass at most.
template <typename Product, int kStages, int kMost>
__global__ void __launch_bounds__(kThreads, 1) experts_kernel(const __grid_constant__ ExpertsArgs a) {
    extern __shared__ __align__(16) uint8_t shared[];
    const Layout at(a.experts, a.tokens, a.top_k, a.k, a.tiles, a.passes_rows, Product::kPairs, kStages);
    Head* const head = reinterpret_cast<Head*>(shared);
    unsigned long long* const masks = reinterpret_cast<unsigned long long*>(shared + at.masks);
    float* const weights = reinterpret_cast<float*>(shared + at.weights);
    uint16_t* const ids = reinterpret_cast<uint16_t*>(shared + at.ids);
    uint32_t* const list = reinterpret_cast<uint32_t*>(shared + at.list);
    uint16_t* const queue = reinterpret_cast<uint16_t*>(shared + at.queue);
    uint8_t* const acts = shared + at.acts;
    const int warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id()), g = lane >> 2, t = lane & 3;
    float4* const scales = reinterpret_cast<float4*>(shared + at.scales) + warp * kUnitRows;
    uint8_t* const own = shared + at.stages + warp * kStages * kStageBytes;
    const uint8_t *stage = own, *const last_stage = own + kStages * kStageBytes;

    // The second kernel starts when every CTA of the first has passed its wait: what came before the call is complete.
    if (!Product::kPairs) grid_wait_prerequisites();
    grid_launch_dependents();
    route(a, head, masks, weights, ids, list, at.list_size);
    Rounds round(range_start(head, a.tiles, blockIdx.x), range_start(head, a.tiles, blockIdx.x + 1), a.tiles, (a.k + kSlice - 1) / kSlice);
    const Pairs pairs{list, at.list_size, head->narrow};
    Stream<Product, kStages> stream(a, pairs, smem_addr(own), round);
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) stream.ask();
    if (Product::kPairs) grid_wait_prerequisites();
    if (Product::kPairs && head->pairs == 0)   // nobody chose anything
        for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < static_cast<int64_t>(a.tokens) * a.dim;
             i += static_cast<int64_t>(gridDim.x) * kThreads)
            a.y[i / a.dim * a.ldy + i % a.dim] = 0;

    const int pitch = Layout::pitch(a.k), low = a.passes_rows * pitch;
    const bool all = !Product::kPairs && a.tokens <= a.passes_rows;
    int pair = -1;
    while (round.advance()) {
        if (round.pair != pair) {
            stage_rows<Product>(a, head, acts, masks, weights, ids, pairs[round.pair], all, all && pair >= 0);
            pair = round.pair;
        }
        const bool wide = kMost > 1 && head->wide != 0;
        float acc[2][kMost][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < kMost; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;
        const uint8_t* x = acts + g * pitch + t * 16 + round.slice * (kSlice * 2);
#pragma unroll 1
        for (int i = round.slice; i < round.last; ++i) {
            copies_wait<kStages - 1>();
            __syncwarp();
            if (wide) multiply<kMost, Product::kPairs>(stage, scales, x, pitch, low, acc);
            else multiply<1, Product::kPairs>(stage, scales, x, pitch, low, acc);
            __syncwarp();
            stream.ask();
            x += kSlice * 2;
            stage += kStageBytes;
            if (stage == last_stage) stage = own;
        }
        const int cols = wide ? kMost : 1;
        // A unit's first warp gets what the others have: at once, or in halves where 16 columns leave room for 8 warps' sums.
        float* const sums = reinterpret_cast<float*>(shared + at.sums) + lane;
#pragma unroll 1
        for (int span = round.parts; span > 1;) {
            const int keep = wide ? span / 2 : 1, first = (warp / round.parts) * (span - keep);
            __syncthreads();   // what was here before has been added up
            if (round.part >= keep && round.part < span)
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < kMost; ++n)
                        if (n < cols)
#pragma unroll
                            for (int i = 0; i < 4; ++i) sums[(((first + round.part - keep) * cols + n) * 8 + m * 4 + i) * 32] = acc[m][n][i];
            __syncthreads();
            if (round.part < keep)
#pragma unroll 1
                for (int p = round.part + keep; p < span; p += keep)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < kMost; ++n)
                            if (n < cols)
#pragma unroll
                                for (int i = 0; i < 4; ++i) acc[m][n][i] += sums[(((first + p - keep) * cols + n) * 8 + m * 4 + i) * 32];
            span = keep;
        }
        if (round.part != 0) continue;
        finish<kMost>(Product(), a, head, queue, round.unit - round.pair * a.tiles, cols, acc);
    }
    copies_wait<0>();
    if (Product::kPairs) {
        __syncthreads();
        join(a, head, queue, weights);
    }
}

// Sets passes and stages for the kernel of `a`, and gives its shared memory, or 0 where it does not fit.
int shape(ExpertsArgs* a, bool pairs) {
    for (int cols = a->tokens <= 8 ? 1 : 2; cols >= 1; --cols) {
        a->passes_rows = 8 * cols;
        for (a->stages = 4; a->stages >= 2; a->stages -= 2) {
            const Layout l(a->experts, a->tokens, a->top_k, a->k, a->tiles, a->passes_rows, pairs, a->stages);
            if (l.total <= kSharedMost) return l.total;
        }
    }
    return 0;
}

inline int tiles_of(int columns, bool pairs) { return (pairs ? 4 : 8) * ((columns + 127) / 128); }

template <typename Product>
cudaError_t launch(ExpertsArgs a, int rows, int k, int sms, cudaStream_t stream) {
    a.rows = rows;
    a.k = k;
    a.tiles = tiles_of(Product::kPairs ? a.dim : a.inner, Product::kPairs);
    const int smem = shape(&a, Product::kPairs);
    if (smem == 0) return cudaErrorInvalidValue;
    const auto kernel = a.passes_rows == 8 ? (a.stages == 4 ? experts_kernel<Product, 4, 1> : experts_kernel<Product, 2, 1>)
                                           : (a.stages == 4 ? experts_kernel<Product, 4, 2> : experts_kernel<Product, 2, 2>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedMost);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
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

// Sizes that the kernels take: what they need of shared memory decides.
bool sizes_ok(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t inner) {
    if (tokens < 0 || tokens > MXFP4_EXPERTS_MAX_TOKENS || experts < 1 || experts > MXFP4_MAX_GROUPS || top_k < 1 ||
        top_k > MXFP4_EXPERTS_MAX_TOP_K || top_k > experts || dim < 1 || dim > 65536 || inner < 1 || inner > 65536)
        return false;
    ExpertsArgs a = {};
    a.experts = static_cast<int32_t>(experts);
    a.tokens = static_cast<int32_t>(tokens > 0 ? tokens : 1);
    a.top_k = static_cast<int32_t>(top_k);
    a.k = static_cast<int32_t>(dim);
    if (shape(&a, false) == 0) return false;
    a.k = static_cast<int32_t>(inner);
    a.tiles = tiles_of(static_cast<int>(dim), true);
    return shape(&a, true) != 0;
}

int64_t counters_bytes(int64_t dim) { return align256((dim + 127) / 128 * 16); }

}  // namespace
}  // namespace mxfp4

extern "C" {

mxfp4_status mxfp4_experts_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k, int64_t dim, int64_t inner, size_t* bytes) {
    if (!mxfp4::sizes_ok(tokens, experts, top_k, dim, inner) || bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
    *bytes = static_cast<size_t>(mxfp4::counters_bytes(dim) + mxfp4::align256(4 * tokens * top_k * inner) +
                                 mxfp4::align256(4 * tokens * top_k * dim));
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
    a.done = reinterpret_cast<uint32_t*>(w);
    a.h = reinterpret_cast<float*>(w + mxfp4::counters_bytes(dim));
    a.part = reinterpret_cast<float*>(w + mxfp4::counters_bytes(dim) + mxfp4::align256(4 * tokens * top_k * inner));
    a.y = static_cast<uint16_t*>(y);
    a.ldy = tokens > 1 ? ldy : 0;
    a.tokens = static_cast<int32_t>(tokens);
    a.experts = static_cast<int32_t>(experts);
    a.top_k = static_cast<int32_t>(top_k);
    a.dim = static_cast<int32_t>(dim);
    a.inner = static_cast<int32_t>(inner);
    a.logits_f32 = flags & MXFP4_EXPERTS_LOGITS_F32 ? 1 : 0;
    a.normalize = flags & MXFP4_EXPERTS_NORMALIZE ? 1 : 0;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.q = static_cast<const uint8_t*>(up_q);
    a.s = static_cast<const uint8_t*>(up_s);
    if (mxfp4::launch<mxfp4::Up>(a, 2 * a.inner, a.dim, sms, s) != cudaSuccess) return MXFP4_ERR_CUDA;
    a.q = static_cast<const uint8_t*>(down_q);
    a.s = static_cast<const uint8_t*>(down_s);
    return mxfp4::launch<mxfp4::Down>(a, a.dim, a.inner, sms, s) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

}  // extern "C"
