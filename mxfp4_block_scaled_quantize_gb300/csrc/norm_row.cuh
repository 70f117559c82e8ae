// norm_row.cuh -- what the layer norm's passes share: a thread's part of a row, and sums over a row.
#pragma once

#include <cuda_bf16.h>

#include "launch_norm.h"
#include "ptx.cuh"

namespace mxfp4 {

// Two fp32 in one instruction each.
__device__ __forceinline__ uint64_t pack2(float2 v) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(v.x), "f"(v.y));
    return p;
}
__device__ __forceinline__ float2 unpack2(uint64_t p) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint64_t both(float v) { return pack2(make_float2(v, v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// A row, and a thread's place in it.  shift: kShifted rows, elements by which a row starts behind a multiple of 16 bytes.
struct RowShape {
    int dim, t, threads, shift;
};

// A thread's 8 kGroups elements of a row, zeros outside it.
//   kWide     groups of 8 consecutive elements, one or two 16-byte accesses each: pitches and dim are multiples of 8, and
//             every address of 16 bytes
//   kShifted  the same at the multiples of 16 bytes around a row of bf16 that starts behind one, in its slot of the ring: a
//             thread's columns then go by the row's shift, which is that of every a.period-th row, and which all of a CTA's
//             rows have in common.  Groups that reach over the row's ends are masked, and stored element by element.
//   kSingle   pairs of bf16, in one access where the row starts at a multiple of 4 bytes, or single fp32: where x, y and dy
//             are not shifted alike
template <bool kF32, NormAccess kAccess, int kGroups>
struct RowPart {
    static constexpr bool kWide = kAccess == kNormWide, kShifted = kAccess == kNormShifted;
    static constexpr int kElements = 8 * kGroups;
    static constexpr int kPairs = kElements / 2;
    static constexpr int kWords = kElements / (kF32 ? 1 : 2);
    static constexpr int kTurn = kWide || kShifted ? 8 : kF32 ? 1 : 2;   // neighbours that a thread takes together
    uint32_t w[kWords];

    __device__ __forceinline__ static int column(int k, const RowShape& s) {
        return ((k / kTurn) * s.threads + s.t) * kTurn + k % kTurn - (kShifted ? s.shift : 0);
    }
    __device__ __forceinline__ static bool inside(int k, const RowShape& s) {
        return kShifted ? static_cast<unsigned>(column(k, s)) < static_cast<unsigned>(s.dim) : column(k, s) < s.dim;
    }
    // kShifted: s, for masks that are worked out where a group needs them.  Those of 32 elements, kept in registers for all rows, spill:
    // 8192 rows of 4100 forward 57 us, 39 so; 16 elements' are kept (backward 69 us so, 68 kept; 8192 of 1001 forward 12.9 and 12.7).
    __device__ __forceinline__ static RowShape afresh(RowShape s) {
        if (kGroups > 2) asm volatile("" : "+r"(s.t));
        return s;
    }
    // kShifted: is all of group j inside.
    __device__ __forceinline__ static bool whole(int j, const RowShape& s) {
        const int c = column(8 * j, s);
        return c >= 0 && c + 8 <= s.dim;
    }

    // kPadded: the bytes around the row, up to multiples of 16, may be read (its slot in shared memory).
    template <bool kPadded = false>
    __device__ __forceinline__ void load(const void* row, const RowShape& s) {
        static_assert(!kShifted || (kPadded && !kF32), "shifted rows: bf16, from the ring");
        const uint8_t* const p = static_cast<const uint8_t*>(row);
        if (kWide || kShifted) {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                constexpr int kLoads = kF32 ? 2 : 1;
                const bool some = kShifted ? column(8 * j, s) > -8 && column(8 * j, s) < s.dim : inside(8 * j, s);
#pragma unroll
                for (int h = 0; h < kLoads; ++h) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (some) v = reinterpret_cast<const uint4*>(p + static_cast<int64_t>(column(8 * j, s)) * (kF32 ? 4 : 2))[h];
                    uint32_t* const d = w + (j * kLoads + h) * 4;
                    d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
                }
                if (kShifted && !whole(j, s)) {
                    const RowShape own = afresh(s);
#pragma unroll
                    for (int k = 8 * j; k < 8 * j + 8; ++k)
                        if (!inside(k, own)) w[k >> 1] &= k & 1 ? 0xFFFFu : 0xFFFF0000u;
                }
            }
        } else if (kF32) {
#pragma unroll
            for (int k = 0; k < kElements; ++k) {
                w[k] = 0u;
                if (inside(k, s)) w[k] = reinterpret_cast<const uint32_t*>(p)[column(k, s)];
            }
        } else if ((reinterpret_cast<uintptr_t>(p) & 3u) == 0) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const int c = column(2 * i, s);
                w[i] = 0u;
                if (c + (kPadded ? 0 : 1) < s.dim) w[i] = *reinterpret_cast<const uint32_t*>(p + 2 * c);
                else if (c < s.dim) w[i] = *reinterpret_cast<const uint16_t*>(p + 2 * c);
                if (kPadded && c + 1 >= s.dim) w[i] &= 0xFFFFu;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const int c = column(2 * i, s);
                const uint16_t* const q = reinterpret_cast<const uint16_t*>(p) + c;
                uint32_t lo = 0u, hi = 0u;
                if (c < s.dim) lo = q[0];
                if (c + 1 < s.dim) hi = q[1];
                w[i] = lo | hi << 16;
            }
        }
    }
    // Elements 2i and 2i + 1.
    __device__ __forceinline__ uint64_t pair(int i) const {
        if (kF32) return pack2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])));
        return pack2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)));
    }
    // v for each of the two, zero behind the row's end.
    __device__ __forceinline__ static uint64_t within(float v, int i, const RowShape& s) {
        if (kWide) return both(inside(2 * i, s) ? v : 0.0f);
        return pack2(make_float2(inside(2 * i, s) ? v : 0.0f, inside(2 * i + 1, s) ? v : 0.0f));
    }
    // kShifted: zeros outside the row.  Only groups over its ends take the masks.
    __device__ __forceinline__ static void clear(uint64_t* v, const RowShape& s) {
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
            if (whole(j, s)) continue;
            const RowShape own = afresh(s);
#pragma unroll
            for (int i = 4 * j; i < 4 * j + 4; ++i) {
                const float2 f = unpack2(v[i]);
                v[i] = pack2(make_float2(inside(2 * i, own) ? f.x : 0.0f, inside(2 * i + 1, own) ? f.y : 0.0f));
            }
        }
    }
    // The pairs v, each element rounded once to the row's type, to the row's elements.
    __device__ __forceinline__ static void store(void* row, const uint64_t* v, const RowShape& s) {
        uint8_t* const p = static_cast<uint8_t*>(row);
        if (kWide || kShifted) {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                float2 f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = unpack2(v[4 * j + i]);
                if (kShifted && !whole(j, s)) {
                    const RowShape own = afresh(s);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (!inside(8 * j + k, own)) continue;
                        const float e = k & 1 ? f[k >> 1].y : f[k >> 1].x;
                        reinterpret_cast<__nv_bfloat16*>(p)[column(8 * j + k, own)] = __float2bfloat16_rn(e);
                    }
                    continue;
                }
                if (!kShifted && !inside(8 * j, s)) continue;
                if (kF32) {
                    float4* const d = reinterpret_cast<float4*>(p + 4 * static_cast<int64_t>(column(8 * j, s)));
                    d[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
                    d[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
                } else {
                    uint32_t h[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) h[i] = to_bf16(f[i]);
                    *reinterpret_cast<uint4*>(p + 2 * static_cast<int64_t>(column(8 * j, s))) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        } else if (kF32) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float2 f = unpack2(v[i]);
                if (inside(2 * i, s)) reinterpret_cast<float*>(p)[column(2 * i, s)] = f.x;
                if (inside(2 * i + 1, s)) reinterpret_cast<float*>(p)[column(2 * i + 1, s)] = f.y;
            }
        } else {
            const bool together = (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const int c = column(2 * i, s);
                const uint32_t h = to_bf16(unpack2(v[i]));
                uint16_t* const q = reinterpret_cast<uint16_t*>(p) + c;
                if (together && c + 1 < s.dim) {
                    *reinterpret_cast<uint32_t*>(q) = h;
                } else {
                    if (c < s.dim) q[0] = static_cast<uint16_t>(h);
                    if (c + 1 < s.dim) q[1] = static_cast<uint16_t>(h >> 16);
                }
            }
        }
    }
    __device__ __forceinline__ static uint32_t to_bf16(float2 f) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
};

// A thread's part of a vector of fp32 or bf16, as pairs in the places of Part, zero behind the row's end.
template <bool kF32, NormAccess kAccess, int kGroups>
__device__ __forceinline__ void load_vector(const void* v, int64_t at, bool f32, bool wide, const RowShape& s, uint64_t* f) {
    using Part = RowPart<kF32, kAccess, kGroups>;
    if (kAccess == kNormWide && wide) {
        if (f32) {
            RowPart<true, kNormWide, kGroups> p;
            p.load(static_cast<const float*>(v) + at, s);
#pragma unroll
            for (int i = 0; i < Part::kPairs; ++i) f[i] = p.pair(i);
        } else {
            RowPart<false, kNormWide, kGroups> p;
            p.load(static_cast<const uint16_t*>(v) + at, s);
#pragma unroll
            for (int i = 0; i < Part::kPairs; ++i) f[i] = p.pair(i);
        }
        return;
    }
    if constexpr (Part::kShifted) {
        // One branch for the type and all loads under way together: 100 rows of 5001 forward 4.8 us, 5.3 as below.  (Single accesses
        // of fp32 lost by it: 8192 rows of 4001 99 us, 44 as below, with as many registers.)
        const RowShape own = Part::afresh(s);
        uint32_t w[Part::kElements];
#pragma unroll
        for (int k = 0; k < Part::kElements; ++k) w[k] = 0u;
        if (f32) {
            const uint32_t* const p = static_cast<const uint32_t*>(v) + at;
#pragma unroll
            for (int k = 0; k < Part::kElements; ++k)
                if (Part::inside(k, own)) w[k] = p[Part::column(k, own)];
        } else {
            const uint16_t* const p = static_cast<const uint16_t*>(v) + at;
#pragma unroll
            for (int k = 0; k < Part::kElements; ++k)
                if (Part::inside(k, own)) w[k] = static_cast<uint32_t>(p[Part::column(k, own)]) << 16;
        }
#pragma unroll
        for (int i = 0; i < Part::kPairs; ++i) f[i] = pack2(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])));
        return;
    }
    auto one = [&](int k) {
        if (!Part::inside(k, s)) return 0.0f;
        const int64_t i = at + Part::column(k, s);
        return f32 ? static_cast<const float*>(v)[i] : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(v)[i]) << 16);
    };
#pragma unroll
    for (int i = 0; i < Part::kPairs; ++i) f[i] = pack2(make_float2(one(2 * i), one(2 * i + 1)));
}

// The columns that a row's threads have to cover: a shifted row's first group starts before it.
inline int columns_of(const NormArgs& a) { return a.dim + (a.access == kNormShifted ? 7 : 0); }

// Threads of a CTA that has a row to itself.
inline int row_threads(int columns, int groups) { return ((columns + 8 * groups - 1) / (8 * groups) + 31) / 32 * 32; }

// How a kernel takes its rows: one a warp, straight into registers; or one a CTA, through a
// ring of rows in shared memory that bulk copies fill ahead of it.
enum RowMode { kWarpRow, kRingRow };

// The ring: `stages` slots of a row's bytes, a barrier each.  Thread 0 fills a slot again once every thread has
// its part of it in registers, which a barrier of the row's sums tells it.  A wait that runs out is
// recorded, no slot is filled any more, and the rows go on with what the slots hold: no thread is left
// waiting for another.
struct RowRing {
    uint64_t full[kNormStages];
    int abort;
};

// How a row lies in its slot.  Bulk copies move whole 16 bytes: a row that does not start or end at a
// multiple of 16 comes with what lies around it in its 16 bytes, which belongs to the rows beside it; the first and the
// last row have no such neighbour, and the threads copy them (`edge`).
template <bool kWide>
__device__ __forceinline__ bool ring_edge(int64_t row, int64_t rows) {
    return !kWide && (row == 0 || row == rows - 1);
}

// Bytes of a slot's row of `bytes`.
template <bool kWide>
__host__ __device__ __forceinline__ uint32_t ring_bytes(uint32_t bytes) {
    return kWide ? bytes : ((bytes + 15u) & ~15u) + 16u;
}

template <bool kWide>
__device__ __forceinline__ uint32_t ring_skew(const uint8_t* row) {
    return kWide ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 15u;
}

// Bytes that the copy of a row of `bytes` moves, and the copy.
template <bool kWide>
__device__ __forceinline__ uint32_t ring_moved(const uint8_t* row, uint32_t bytes) {
    return kWide ? bytes : (ring_skew<kWide>(row) + bytes + 15u) & ~15u;
}

template <bool kWide>
__device__ __forceinline__ void ring_copy(uint32_t to, const uint8_t* row, uint32_t bytes, uint32_t bar) {
    bulk_load(to, row - ring_skew<kWide>(row), ring_moved<kWide>(row, bytes), bar);
}

__device__ __forceinline__ void ring_init(RowRing* r, int count, int stages) {
    if (static_cast<int>(threadIdx.x) < count) {
        for (int i = 0; i < stages; ++i) mbar_init(smem_addr(&r[threadIdx.x].full[i]), 1);
        r[threadIdx.x].abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
}

// A row's threads meet: all of a CTA's, or one of its teams' of `threads`.
template <bool kTeams>
__device__ __forceinline__ void row_meet(int team, int threads) {
    if (kTeams) named_barrier(1 + team, threads);
    else __syncthreads();
}

__device__ __forceinline__ void ring_wait(RowRing& r, int slot, uint32_t phase, uint32_t* err) {
    mbar_wait(smem_addr(&r.full[slot]), phase, err, kErrNorm, &r.abort);
}

template <bool kF32>
struct Element { using Type = uint16_t; };
template <>
struct Element<true> { using Type = uint32_t; };

// An edge row into its slot, by thread t of `threads`; a barrier of theirs is to follow.
template <bool kF32>
__device__ __forceinline__ void ring_fill(uint8_t* to, const uint8_t* row, int dim, int t, int threads) {
    using T = typename Element<kF32>::Type;
    constexpr int kTogether = 16;   // loads under way
    const T* const from = reinterpret_cast<const T*>(row);
#pragma unroll 1
    for (int i = t; i < dim; i += kTogether * threads) {
        T v[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) v[k] = from[min(i + k * threads, dim - 1)];
#pragma unroll
        for (int k = 0; k < kTogether; ++k)
            if (i + k * threads < dim) reinterpret_cast<T*>(to)[i + k * threads] = v[k];
    }
    fence_proxy_async_smem();   // a copy writes the slot next
}

// Thread 0, before it ends: copies that a wait gave up on may still be on their way.
__device__ __forceinline__ void ring_drain(RowRing& r, int stages, int issued) {
    if (*static_cast<volatile int*>(&r.abort) == 0) return;   // every copy has been waited for
    for (int i = issued < stages ? 0 : issued - stages; i < issued; ++i)
        mbar_wait_quiet(smem_addr(&r.full[i % stages]), (i / stages) & 1, kWaitLimitNs);
}

template <int kLanes>
__device__ __forceinline__ uint64_t lanes_sum2(uint64_t v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v = add2(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

template <int kLanes>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// Two sums over the row's threads, in all of them and in the same order in each.  A row of several warps, of
// kWarps at most, goes through `shared`, which two calls in a row do not share: one barrier a call.
template <RowMode kMode, int kWarps, bool kTeams>
__device__ __forceinline__ float2 row_sum2(uint64_t v, uint64_t* shared, int t, int team, int threads) {
    v = lanes_sum2<32>(v);
    if (kMode == kWarpRow) return unpack2(v);
    if (lane_id() == 0) shared[t >> 5] = v;
    row_meet<kTeams>(team, threads);
    const int i = static_cast<int>(lane_id()) & (kWarps - 1);
    return unpack2(lanes_sum2<kWarps>(i < threads >> 5 ? shared[i] : 0ull));
}

}  // namespace mxfp4
