// gemm_grouped.cu -- the block-scaled MXF4 products of a linear grouped by expert, on CTA pairs
// (tcgen05 cta_group::2), all groups in one launch.
//
// Three forms over the grouped blobs (quantize_grouped.cu), group e of m_e rows starting at
// row o_e of G and at padded row P_e (a multiple of 128):
//   forward  C[o_e + i, n] = sum_k W_e[n, k] X[i, k]     row blobs of W and X
//   dgrad    C[o_e + i, k] = sum_n W_e[n, k] dY[i, n]    col blob of W, row blob of dY
//   wgrad    C[e, n, k]    = sum_t dY[t, n] X[t, k]      col blobs, over the padded rows t of group e
// so in every form each output tile is an ordinary K-packed product whose operands start
// somewhere inside the blobs: at a row, or at a multiple of 128 along the packed axis.  One
// tensor map per operand (and box height) covers all groups, and a tile is a pair of
// coordinates into each.
//
// In forward and dgrad the rows of W are the MMA's M and the tokens its N: W's tiles of 256 rows
// are always whole, and the tokens of a group, of which there may be one or ten thousand, are
// cut into tiles of 384 and a last one of any multiple of 32, which takes that much less of the
// tensor pipe and of the operand bytes, the scarcest thing here.  (With the tokens as M, in tiles of
// 256 rows, forward took, in us: 64 groups of 384 tokens on average, 1408 x 2048, 57.4, and 55.3 here;
// 8 groups of 2048, 8192 x 2048, 133.1 and 112.6; 64 groups of 4, 2048 x 2048, 38.9 and 32.8; 8 single
// tokens 14.3 both.)  The accumulator then
// holds C transposed, and the epilogue turns 32 x 32 pieces round in shared memory.  What a tile
// holds past its group are the next group's rows: their products are never stored, and an
// FP4 product has no NaN to spread.  A group without rows has no tile in forward and dgrad,
// and tiles of zeros in wgrad, which no MMA touches.
//
// TMEM holds 384 accumulator columns.  Tiles take them from the low and the high end in turn, so
// that the read-out of one hides behind the MMAs of the next wherever both fit.  (Working a tile
// of 384 columns off as 256 and 128, which always fit, lost 20 to 30 %: a K step then costs
// nearly as much for a third or two thirds of the work.)
//
// The few-token instances (launches whose groups have some 96 tokens or fewer on average) have
// tiles of up to 128 tokens and seven stages in place of four: they are bound by the stream of
// W, which needs the more bytes in flight.  (64 groups of 8 tokens, 2048 x 2048: 38.9 us, 45.1 by the
// other instance; of 96 tokens 41.0 and 47.1; of 192, two tiles, 55.3 and 49.2.)
//
// Roles as in the pair kernel (gemm_pair.cu).  The clusters take the tiles round-robin (the token
// tiles of one W tile in turn, then the next W tile), each wave rotated by one cluster, or clusters
// would keep meeting tiles of one size: neighbours then read the same W tile, or the same
// tokens, at the same time.  (A contiguous run of tiles for each cluster, balanced by cost, took 178 us
// where this took 125: forward of 32 groups of 512 tokens on average, 4096 x 4096.)  The MMA warp must not touch shared memory with MMAs in flight, so the
// waiter hands it what it has to know of a tile with every stage, as the count of a barrier
// reduction.
#include <cuda_bf16.h>

#include <type_traits>

#include "epilogue.cuh"
#include "group_table.cuh"
#include "launch.h"
#include "pair_common.cuh"
#include "ptx.cuh"

namespace mxfp4 {
namespace {

constexpr int BKB = 128;                  // bytes of K per stage (256 FP4 elements)
constexpr int kABytes = 128 * BKB;        // this CTA's 128 rows of the M operand
constexpr int kSfaBytes = 2 * 512;        // 2 scale atoms of this CTA's M rows
constexpr int kEpi0 = 3;                  // warps 0 producer, 1 MMA, 2 MMA waiter
constexpr int kEpiWarps = 12;             // 4 lane quarters x 3 column groups
constexpr int kThreads = (kEpi0 + kEpiWarps) * 32;
constexpr uint32_t kBarHandoff = 1;
constexpr uint32_t kBarEpilogue = 2;
constexpr uint32_t kTmemCols = 512;

template <bool kFew>
struct Cfg {
    static constexpr int kMaxN = kFew ? 128 : 384;       // columns of a tile, and of the accumulators together: x 2, x 1
    static constexpr int kStages = kFew ? 7 : 4;
    static constexpr int kGroups = kMaxN / 128;          // 128-row scale groups of the N operand
    static constexpr int kBBytes = kMaxN / 2 * BKB;      // this CTA's half of the tile's N rows
    static constexpr int kSfbBytes = kGroups * 2 * 512;
    static constexpr uint32_t kAccCols = kFew ? 256 : 384;
    static constexpr uint32_t kSfTmemPerStage = 8 + 8 * kGroups;   // per atom: 4 columns a group, A's first
    static_assert(kAccCols + kStages * kSfTmemPerStage <= kTmemCols, "TMEM budget");
};

template <bool kFew>
struct GroupedSmem {
    using C = Cfg<kFew>;
    uint8_t a[C::kStages][kABytes];       // 1024-byte aligned (128-byte swizzle atoms)
    uint8_t b[C::kStages][C::kBBytes];    // a tile's columns 0 .. 255, then the others at 16 KB
    uint8_t out[kEpiWarps][kOutBytes];
    uint8_t sfa[C::kStages][kSfaBytes];
    uint8_t sfb[C::kStages][C::kSfbBytes];
    uint64_t full[C::kStages];            // used in the leader: both CTAs' bytes
    uint64_t empty[C::kStages];           // each CTA: the leader's MMA commit
    uint64_t tmem_full[2];                // each CTA, per side: the leader's commit after a tile
    uint64_t tmem_empty[2];               // used in the leader: 2 x kEpiWarps arrivals
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    int32_t tiles_n[kMaxGroups + 1];      // N tiles of the groups before
    GroupTable table;
};

struct Tile {
    int e, mt, n0;        // group, 256-row tile of the M operand, first row of the N operand in the group
    int columns;          // accumulator columns: rows of the N operand, rounded up to 32; 0: no tile
    int atoms;            // K atoms (128 elements each)
};

__device__ __forceinline__ int tiles_in(int rows, int width) {
    int rest;
    return small_div(rows + width - 1, width, &rest);
}

template <bool kWgrad, bool kFew>
__device__ __forceinline__ Tile tile_at(int i, const GroupedGemmArgs& g, const GroupedSmem<kFew>& sm) {
    Tile r;
    int rest, nt;
    r.e = find_group(sm.tiles_n, g.groups, small_div(i, g.tiles_m, &rest));
    r.mt = small_div(i - sm.tiles_n[r.e] * g.tiles_m, sm.tiles_n[r.e + 1] - sm.tiles_n[r.e], &nt);
    r.n0 = nt * g.width;
    r.atoms = kWgrad ? sm.table.tiles[r.e + 1] - sm.table.tiles[r.e] : g.atoms;
    const int rows = kWgrad ? g.n_cols : sm.table.start[r.e + 1] - sm.table.start[r.e];
    r.columns = min(g.width, (rows - r.n0 + 31) & ~31);
    return r;
}

// The tiles of a cluster, as one warp walks them.  Finding a tile takes over a thousand cycles
// (divisions, a search in shared memory), so the lanes find the tiles of 32 waves at once, and
// each tile is then a few shuffles.
template <bool kWgrad, bool kFew>
struct Tiles {
    const GroupedGemmArgs& g;
    const GroupedSmem<kFew>& sm;
    int wave = 0;
    Tile mine{};   // of wave (wave & ~31) + lane

    __device__ __forceinline__ Tiles(const GroupedGemmArgs& g_, const GroupedSmem<kFew>& sm_) : g(g_), sm(sm_) {}

    // The next tile; columns == 0 after the last.  The whole warp.
    __device__ __forceinline__ Tile next() {
        if ((wave & 31) == 0) {
            const int nclusters = static_cast<int>(gridDim.x >> 1), cluster = static_cast<int>(blockIdx.x >> 1);
            const int w = wave + static_cast<int>(lane_id()), total = sm.tiles_n[g.groups] * g.tiles_m;
            int turn;
            small_div(cluster + w, nclusters, &turn);
            mine.columns = 0;
            // (w nclusters < total for every wave up to the last, so neither product leaves 32 bits)
            if (w <= total / nclusters && w * nclusters + turn < total) mine = tile_at<kWgrad, kFew>(w * nclusters + turn, g, sm);
            __syncwarp();
        }
        const int from = wave++ & 31;
        Tile r;
        r.e = __shfl_sync(0xFFFFFFFFu, mine.e, from);
        r.mt = __shfl_sync(0xFFFFFFFFu, mine.mt, from);
        r.n0 = __shfl_sync(0xFFFFFFFFu, mine.n0, from);
        r.columns = __shfl_sync(0xFFFFFFFFu, mine.columns, from);
        r.atoms = kWgrad ? __shfl_sync(0xFFFFFFFFu, mine.atoms, from) : g.atoms;
        return r;
    }
};

// A value that is the same in all lanes, for the compiler to know it too.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }

// Index of the lowest box of 16 << i rows that holds `rows` rows.
__device__ __forceinline__ int box_of(int rows) { return rows <= 16 ? 0 : rows <= 32 ? 1 : rows <= 64 ? 2 : 3; }

template <bool kWgrad, bool kF32, bool kFew>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ GroupedGemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    using C = Cfg<kFew>;
    constexpr int kStages = C::kStages;
    GroupedSmem<kFew>& sm = *reinterpret_cast<GroupedSmem<kFew>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                                  ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const int rank = static_cast<int>(cluster_cta_rank());
    const bool leader = rank == 0;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_addr(&sm.tmem_full[b]), 1);
            mbar_init(smem_addr(&sm.tmem_empty[b]), 2 * kEpiWarps);
        }
        mbar_init(smem_addr(&sm.drain), 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&sm.tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    // Where nothing in flight writes the offsets, no role waits for the launch ahead but the producer,
    // before its first copies (that launch has no part in C either).
    if (!g.early_offsets) grid_wait_prerequisites();
    grid_launch_dependents();
    if (warp == 2)
        build_group_table(sm.table, g.offsets, g.groups, g.rows, g.err, sm.tiles_n,
                          [&](int m) { return tiles_in(kWgrad ? g.n_cols : m, g.width); });
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers exist before anything signals across
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        // The whole warp walks the tiles, lane 0 waits and copies.
        if (lane == 0) {
            prefetch_tensormap(&g.amap);
            prefetch_tensormap(&g.sfamap);
            prefetch_tensormap(&g.sfbmap);
            for (int i = 0; i < (kFew ? 3 : 4); ++i) prefetch_tensormap(&g.bmap[i]);
        }
        const uint64_t pol = l2_policy_evict_last();
        const uint32_t full0 = cluster_map(smem_addr(&sm.full[0]), 0);
        // What a tile's copies share.  Coordinates along the packed axis in bytes (scales: 8-byte
        // units).  The N operand's first 256 rows are one MMA's, the rest another's; a CTA holds
        // half of each.
        struct Copies {
            int m_x, m_row, m_group, n_x, n_row, n_row1, n_group, half1;
            const CUtensorMap *n_map, *n_map1;
            uint32_t bytes;
        };
        auto copies_of = [&](const Tile& t) {
            Copies c;
            const int half0 = min(t.columns, 256) / 2;
            const int first = sm.table.start[t.e], padded = sm.table.tiles[t.e];
            c.half1 = kFew ? 0 : (t.columns - 2 * half0) / 2;
            c.m_x = (kWgrad ? padded : t.e * g.a_step_atoms) * 64;
            c.m_row = (kWgrad ? 0 : t.e * g.a_step_rows) + t.mt * 256 + rank * 128;
            c.m_group = (kWgrad ? 0 : t.e * g.a_step_groups) + 2 * t.mt + rank;
            c.n_x = kWgrad ? padded * 64 : 0;
            c.n_row = (kWgrad ? 0 : first) + t.n0 + rank * half0;
            c.n_row1 = (kWgrad ? 0 : first) + t.n0 + 256 + rank * c.half1;
            c.n_group = (kWgrad ? 0 : padded) + t.n0 / 128;
            c.n_map = &g.bmap[box_of(half0)];
            c.n_map1 = &g.bmap[box_of(c.half1)];
            const int rows = (16 << box_of(half0)) + (c.half1 > 0 ? 16 << box_of(c.half1) : 0);
            c.bytes = 2 * (kABytes + kSfaBytes + C::kSfbBytes + rows * BKB);
            return c;
        };
        auto load_m = [&](const Copies& c, int ks, int s) {
            if (leader) mbar_arrive_expect_tx(smem_addr(&sm.full[s]), c.bytes);
            tma_load_2d_pair(smem_addr(sm.a[s]), &g.amap, c.m_x + ks * BKB, c.m_row, full0 + 8 * s, pol);
            tma_load_2d_pair(smem_addr(sm.sfa[s]), &g.sfamap, c.m_x + ks * 128, c.m_group, full0 + 8 * s, pol);
        };
        auto load_n = [&](const Copies& c, int ks, int s) {
            tma_load_2d_pair(smem_addr(sm.b[s]), c.n_map, c.n_x + ks * BKB, c.n_row, full0 + 8 * s, pol);
            if (!kFew && c.half1 > 0)
                tma_load_2d_pair(smem_addr(sm.b[s]) + 128 * BKB, c.n_map1, c.n_x + ks * BKB, c.n_row1, full0 + 8 * s, pol);
            tma_load_2d_pair(smem_addr(sm.sfb[s]), &g.sfbmap, c.n_x + ks * 128, c.n_group, full0 + 8 * s, pol);
        };
        int it = 0, s = 0, ahead = 0;
        uint32_t ph = 1;
        int ok = 1;
        Tiles<kWgrad, kFew> tiles(g, sm);
        while (ok) {
            const Tile t = tiles.next();
            if (t.columns == 0) break;
            if (lane == 0) {
                const Copies c = copies_of(t);
                const int steps = (t.atoms + 1) >> 1;
                if (g.early_offsets && it == 0) {
                    // the first tile's M operand is on its way before the N operand exists
                    if (g.early_m)
                        for (; ahead < min(steps, kStages); ++ahead) load_m(c, ahead, ahead);
                    grid_wait_prerequisites();
                }
                for (int ks = 0; ks < steps; ++ks, ++it) {
                    if (it >= ahead) {
                        if (!mbar_wait(smem_addr(&sm.empty[s]), ph, g.err, kErrGemmProducer, &sm.abort)) {
                            ok = 0;
                            break;
                        }
                        load_m(c, ks, s);
                    }
                    load_n(c, ks, s);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
        }
        if (lane == 0) grid_wait_prerequisites();   // clusters without a tile too: this grid ends after the one ahead
        // Drain (leader): every armed stage, both CTAs' bytes, has landed.
        if (leader && lane == 0) {
            const int armed = it < kStages ? it : kStages;
            for (int i = 1; i <= armed; ++i) {
                const int j = it - i;
                mbar_wait_quiet(smem_addr(&sm.full[j % kStages]), (j / kStages) & 1, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        if (leader) {
            const int fixed_steps = (g.atoms + 1) >> 1;   // forward, dgrad: of every tile
            int side = 1, ks = 0, s = 0;
            for (;;) {
                // 0: no more, else columns / 32; wgrad: then 1 (more steps follow in the tile), 2 (its
                // last) or 3 (its last, of one atom)
                const int n32 = static_cast<int>(uniform(named_barrier_count(kBarHandoff, 64, false)));
                if (n32 == 0) break;
                int natoms = 2;
                bool last;
                if (kWgrad) {
                    const int u = static_cast<int>(uniform(named_barrier_count(kBarHandoff, 64, false)));
                    last = u > 1;
                    natoms = u == 3 ? 1 : 2;
                } else {
                    last = ks == fixed_steps - 1;
                    natoms = min(2, g.atoms - 2 * ks);
                }
                if (ks == 0) side ^= 1;
                const uint32_t d = tmem + (side ? C::kAccCols - 32 * n32 : 0u);
                const uint32_t sf = tmem + C::kAccCols + s * C::kSfTmemPerStage;
                const uint32_t sfa_s = smem_addr(sm.sfa[0]) + s * kSfaBytes;
                const uint32_t sfb_s = smem_addr(sm.sfb[0]) + s * C::kSfbBytes;
                const uint64_t adesc = smem_desc(smem_addr(sm.a[0]) + s * kABytes, 16, 1024, 2);
                const uint64_t bdesc = smem_desc(smem_addr(sm.b[0]) + s * C::kBBytes, 16, 1024, 2);
                const uint64_t bdesc2 = smem_desc(smem_addr(sm.b[0]) + s * C::kBBytes + 128 * BKB, 16, 1024, 2);
                const uint32_t more = ks != 0;
                // One stage's copies and MMAs, without a branch among them: any there makes the copies
                // wait for the MMAs issued before.
                auto issue = [&](auto atoms_, auto two_) {
                    constexpr int kAtoms = decltype(atoms_)::value;
                    constexpr bool kTwo = decltype(two_)::value;
                    if (elect_one()) {
                        tc_fence_after_sync();
#pragma unroll
                        for (int a = 0; a < kAtoms; ++a) {
                            const uint32_t sfb = sf + 8 + a * 4 * C::kGroups;
                            tc_cp_32x128b_warpx4_pair(sf + a * 4, smem_desc(sfa_s + a * 512, 0, 128, 0));
#pragma unroll
                            for (int gb = 0; gb < (kTwo ? 3 : C::kGroups < 2 ? 1 : 2); ++gb)
                                tc_cp_32x128b_warpx4_pair(sfb + gb * 4, smem_desc(sfb_s + gb * 1024 + a * 512, 0, 128, 0));
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                const int j = 2 * a + jj;
                                tc_mma_mxf4_pair(d, adesc + 2 * j, bdesc + 2 * j, pair_idesc(jj * 2, kTwo ? 256 : 32 * n32),
                                                 sf + a * 4, sfb, j != 0 ? 1u : more);
                                if (kTwo)
                                    tc_mma_mxf4_pair(d + 256, adesc + 2 * j, bdesc2 + 2 * j, pair_idesc(jj * 2, 32 * n32 - 256),
                                                     sf + a * 4, sfb + 8, j != 0 ? 1u : more);
                            }
                        }
                        tc_commit_pair_multicast(smem_addr(&sm.empty[0]) + 8 * s, 3);
                    }
                };
                using One = std::integral_constant<int, 1>;
                using Two = std::integral_constant<int, 2>;
                if (!kFew && n32 > 8) {
                    if (natoms == 2) issue(Two{}, std::integral_constant<bool, !kFew>{});
                    else issue(One{}, std::integral_constant<bool, !kFew>{});
                } else {
                    if (natoms == 2) issue(Two{}, std::false_type{});
                    else issue(One{}, std::false_type{});
                }
                if (last && elect_one()) tc_commit_pair_multicast(smem_addr(&sm.tmem_full[0]) + 8 * side, 3);
                ks = last ? 0 : ks + 1;
                if (++s == kStages) s = 0;
            }
            if (elect_one()) {
                tc_commit_pair_multicast(smem_addr(&sm.drain), 1);
                if (!mbar_wait_quiet(smem_addr(&sm.drain), 0, kWaitLimitNs)) atomicOr(g.err, kErrGemmDrain);
            }
            __syncwarp();
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------------ MMA waiter
        if (leader) {
            int it = 0, tl = 0;
            int before = 0;   // columns of the tile before
            bool ok = true;
            Tiles<kWgrad, kFew> tiles(g, sm);
            while (ok) {
                const Tile t = tiles.next();
                if (t.columns == 0) break;
                const int steps = (t.atoms + 1) >> 1;
                if (steps == 0) continue;
                const int side = tl & 1;
                for (int ks = 0; ks < steps; ++ks, ++it) {
                    int good = 1;
                    if (lane == 0) {
                        // the tile two before was on this side; the one before may reach into it
                        if (ks == 0 && tl > 1)
                            good = mbar_wait(smem_addr(&sm.tmem_empty[side]), ((tl >> 1) - 1) & 1, g.err, kErrGemmMma, &sm.abort);
                        if (good && ks == 0 && tl > 0 && t.columns + before > static_cast<int>(C::kAccCols))
                            good = mbar_wait(smem_addr(&sm.tmem_empty[side ^ 1]), ((tl - 1) >> 1) & 1, g.err, kErrGemmMma,
                                             &sm.abort);
                        if (good)
                            good = mbar_wait(smem_addr(&sm.full[it % kStages]), (it / kStages) & 1, g.err, kErrGemmMma,
                                             &sm.abort);
                    }
                    if (!__shfl_sync(0xFFFFFFFFu, good, 0)) {
                        ok = false;
                        break;
                    }
                    // columns / 32; wgrad: and 1 (more steps follow), 2 (the last) or 3 (the last, one atom)
                    named_barrier_count(kBarHandoff, 64, static_cast<int>(lane) < t.columns / 32);
                    if (kWgrad)
                        named_barrier_count(kBarHandoff, 64,
                                            static_cast<int>(lane) < (ks < steps - 1 ? 1 : (t.atoms & 1) ? 3 : 2));
                }
                before = t.columns;
                ++tl;
            }
            named_barrier_count(kBarHandoff, 64, false);
        }
    } else {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int h = (warp - kEpi0) >> 2;
        const uint32_t obuf = smem_addr(sm.out[warp - kEpi0]);
        const uint64_t pol = l2_policy_evict_normal();
        if (lane == 0 && g.c_tma) prefetch_tensormap(&g.cmap);
        int tl = 0;
        Tiles<kWgrad, kFew> tiles(g, sm);
        while (true) {
            const Tile t = tiles.next();
            if (t.columns == 0) break;
            // This warp's 32-column pieces of the tile: h, h + 3, ..., four at most.
            const int mine = (t.columns / 32 - h + 2) / 3;
            const int m0 = t.mt * 256 + rank * 128 + q * 32;   // of the M operand's rows, in the group
            const int n_end = kWgrad ? g.n_cols : sm.table.start[t.e + 1] - sm.table.start[t.e];   // N operand's rows
            // C's row that m0 (wgrad) or row 0 of the N operand (forward, dgrad) is
            const int64_t base = kWgrad ? static_cast<int64_t>(t.e) * g.m_rows + m0 : sm.table.start[t.e];
            // Stores piece k: x holds this lane's 32 accumulator columns, as bf16 pairs or fp32.
            auto store = [&](int k, const uint32_t (&x)[kF32 ? 32 : 16]) {
                const int n0 = t.n0 + 32 * (h + 3 * k);
                if (k >= mine || m0 >= g.m_rows || n0 >= n_end) return;
                const bool live = m0 + static_cast<int>(lane) < g.m_rows;
                if (kWgrad) {
                    if (g.c_tma && m0 + 32 <= g.m_rows) {
#pragma unroll
                        for (int c = 0; c < (kF32 ? 2 : 1); ++c) {   // 64-byte pieces of a row
                            if (n0 + 16 * c >= n_end) break;
                            if (lane == 0) bulk_wait_read_all();
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                sts128(obuf + swz64(lane, j), x[16 * c + 4 * j], x[16 * c + 4 * j + 1], x[16 * c + 4 * j + 2],
                                       x[16 * c + 4 * j + 3]);
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_2d_hint(&g.cmap, n0 + 16 * c, static_cast<int32_t>(base), obuf, pol);
                                bulk_commit_group();
                            }
                        }
                    } else if (live) {   // a group's last rows, or a pitch that no tensor store takes
                        const int cols = min(n_end - n0, 32);
                        const int64_t at = (base + lane) * g.ldc + n0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            if (j >= cols) break;
                            if (kF32) static_cast<uint32_t*>(g.c)[at + j] = x[j & (kF32 ? 31 : 15)];
                            else static_cast<uint16_t*>(g.c)[at + j] = static_cast<uint16_t>(x[(j >> 1) & 15] >> (16 * (j & 1)));
                        }
                    }
                    return;
                }
                // forward, dgrad: this lane's column of C, accumulator columns = its rows
                if (!kF32 && g.c_tma && n0 + 32 <= n_end) {
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
                    // word i holds tokens 2 i and 2 i + 1 of this lane's column; with its neighbour a
                    // lane makes one row's pair of columns: even lanes token 2 i, odd 2 i + 1
                    const uint32_t at = obuf + (lane & 1u) * kOutRowBytes + ((lane >> 1) & 3u) * 4;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, x[r], 1);
                        sts32(at + swz64(2 * r, lane >> 3),
                              (lane & 1u) ? __byte_perm(other, x[r], 0x7632) : __byte_perm(x[r], other, 0x5410));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d_hint(&g.cmap, m0, static_cast<int32_t>(base + n0), obuf, pol);
                        bulk_commit_group();
                    }
                } else if (live) {
                    // fp32: a row's 32 columns are a line; bf16: the group's last rows, or a pitch that no
                    // tensor store takes
                    const int rows = min(n_end - n0, 32);
                    const int64_t at = (base + n0) * g.ldc + m0 + lane;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (j >= rows) break;
                        if (kF32) static_cast<uint32_t*>(g.c)[at + j * g.ldc] = x[j & (kF32 ? 31 : 15)];
                        else static_cast<uint16_t*>(g.c)[at + j * g.ldc] = static_cast<uint16_t>(x[(j >> 1) & 15] >> (16 * (j & 1)));
                    }
                }
            };
            if (t.atoms == 0) {   // wgrad of a group without rows
                uint32_t x[kF32 ? 32 : 16];
#pragma unroll
                for (int r = 0; r < (kF32 ? 32 : 16); ++r) x[r] = 0u;
#pragma unroll 1
                for (int k = 0; k < mine; ++k) store(k, x);
                continue;
            }
            const int side = tl & 1;
            int okw = 1;
            if (warp == kEpi0 && lane == 0)
                okw = mbar_wait(smem_addr(&sm.tmem_full[side]), (tl >> 1) & 1, g.err, kErrGemmEpilogue, &sm.abort);
            if (!named_barrier_and(kBarEpilogue, kEpiWarps * 32, __shfl_sync(0xFFFFFFFFu, okw, 0) != 0)) break;
            ++tl;
            tc_fence_after_sync();
            const uint32_t taddr =
                tmem + (side ? C::kAccCols - t.columns : 0u) + (static_cast<uint32_t>(q * 32) << 16) + 32 * h;
            // Two pieces at a time (the second of a pair may lie past this warp's last: the first is
            // read again).  The accumulator is released when its last pair is in registers.
            auto read = [&](int k, uint32_t (&f0)[32], uint32_t (&f1)[32]) {
                tc_ld_32x32b_x32(taddr + 96 * k, f0);
                tc_ld_32x32b_x32(taddr + 96 * (k + 1 < mine ? k + 1 : k), f1);
                tc_wait_ld();
            };
            auto release = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_addr(&sm.tmem_empty[side]), 0));
            };
            uint32_t f0[32], f1[32];
            if (kF32) {
#pragma unroll 1
                for (int k = 0; k < 4; k += 2) {
                    if (k < mine) read(k, f0, f1);
                    if (k + 2 >= mine && (k == 0 || mine > 2)) release();
                    if (k >= mine) break;
                    store(k, reinterpret_cast<const uint32_t(&)[kF32 ? 32 : 16]>(f0));
                    store(k + 1, reinterpret_cast<const uint32_t(&)[kF32 ? 32 : 16]>(f1));
                }
            } else {
                // all pieces as bf16 pairs first: the release waits for no store
                uint32_t v[4][kF32 ? 32 : 16];
                auto pack = [&](const uint32_t (&f)[32], uint32_t (&x)[kF32 ? 32 : 16]) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        x[r] = pack_bf16x2(f[2 * r], f[2 * r + 1]);
                        asm volatile("" : "+r"(x[r]));   // before the next pair is read
                    }
                };
                if (mine > 0) {
                    read(0, f0, f1);
                    pack(f0, v[0]);
                    pack(f1, v[1]);
                }
                if (mine > 2) {
                    read(2, f0, f1);
                    pack(f0, v[2]);
                    pack(f1, v[3]);
                }
                release();
#pragma unroll
                for (int k = 0; k < 4; ++k) store(k, v[k]);
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // no CTA leaves or frees TMEM while its peer may still use it
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

size_t smem_bytes(bool few) { return (few ? sizeof(GroupedSmem<true>) : sizeof(GroupedSmem<false>)) + 1024; }
static_assert(sizeof(GroupedSmem<true>) + 1024 <= 232448 && sizeof(GroupedSmem<false>) + 1024 <= 232448,
              "shared memory of a CTA");

}  // namespace

int gemm_grouped_max_clusters() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] > 0) return cached[dev];
    auto kernel = gemm_grouped_kernel<true, true, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(false)) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes(false);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    cached[dev] = n;
    return n;
}

cudaError_t launch_gemm_grouped(const GroupedGemmArgs& a, bool wgrad, bool few, int clusters, cudaStream_t stream) {
    auto kernel = wgrad ? (a.out_f32 ? gemm_grouped_kernel<true, true, false> : gemm_grouped_kernel<true, false, false>)
                  : few ? (a.out_f32 ? gemm_grouped_kernel<false, true, true> : gemm_grouped_kernel<false, false, true>)
                        : (a.out_f32 ? gemm_grouped_kernel<false, true, false> : gemm_grouped_kernel<false, false, false>);
    const size_t smem = smem_bytes(few);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mxfp4
