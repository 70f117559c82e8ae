// gemm_grouped.cu -- the block-scaled MXF4 products of a linear grouped by expert, on CTA pairs
// (tcgen05 cta_group::2), all groups in one launch.
//
// Three forms over the grouped blobs (quantize_grouped.cu), group e of m_e rows starting at
// row o_e of G and at padded row P_e (a multiple of 128):
//   forward  C[o_e + i, n] = sum_k A[i, k] B_e[n, k]     A: row blob of X, B: row blob of W
//   dgrad    C[o_e + i, k] = sum_n A[i, n] B_e[k, n]     A: row blob of dY, B: col blob of W
//   wgrad    C[e, n, k]    = sum_t A[n, t] B[k, t]       A: col blob of dY, B: col blob of X, over
//                                                        the padded rows t of group e
// so in every form each output tile is an ordinary K-packed product whose operands start
// somewhere inside the blobs: at a row (forward, dgrad: A; forward: B), or at a multiple of
// 128 along the packed axis (dgrad: B; wgrad: both).  One tensor map per operand covers all
// groups, and a tile is a pair of coordinates into each.
//
// The kernel is the pair kernel (gemm_pair.cu: roles, barriers, TMEM use) with its tile list
// read off the group table: 256 x 256 tiles, in forward and dgrad the 256-row tiles of each
// group times the column tiles (the row tiles of a group fastest: they share the group's B),
// in wgrad the tiles of every group, with as many K steps as the group has tokens.  A tile's
// rows past its group hold the next group's rows: their products are never stored, and an
// FP4 product has no NaN to spread.  Whole 32-row pieces leave through tensor stores; the
// piece that straddles the group's end is stored row by row.  A group without rows has no
// tile in forward and dgrad, and a tile of zeros in wgrad, which no MMA touches.
#include <cuda_bf16.h>

#include "epilogue.cuh"
#include "group_table.cuh"
#include "launch.h"
#include "pair_common.cuh"
#include "ptx.cuh"

namespace mxfp4 {
namespace {

constexpr int BKB = 128;                  // bytes of K per stage (256 FP4 elements)
constexpr int kStages = 5;
constexpr int kABytes = 128 * BKB;        // this CTA's 128 A rows
constexpr int kBBytes = 128 * BKB;        // this CTA's half of the tile's 256 B rows
constexpr int kSfaBytes = 2 * 512;        // 2 scale atoms of this CTA's rows
constexpr int kSfbBytes = 2 * 2 * 512;    // 2 row groups x 2 atoms
constexpr uint32_t kStageBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
constexpr int kEpi0 = 3;                  // warps 0 producer, 1 MMA, 2 MMA waiter
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpi0 + kEpiWarps) * 32;
constexpr uint32_t kBarHandoff = 1;
constexpr uint32_t kBarEpilogue = 2;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfTmemBase = 256;     // after the accumulator
constexpr uint32_t kSfTmemPerStage = 24;  // per atom: A 4 columns; B 2 groups x 4
static_assert(kSfTmemBase + kStages * kSfTmemPerStage <= kTmemCols, "TMEM budget");

struct GroupedSmem {
    uint8_t a[kStages][kABytes];          // 1024-byte aligned (128-byte swizzle atoms)
    uint8_t b[kStages][kBBytes];
    uint8_t sfa[kStages][kSfaBytes];
    uint8_t sfb[kStages][kSfbBytes];
    uint8_t out[kEpiWarps][kOutBytes];
    uint64_t full[kStages];               // used in the leader: both CTAs' bytes
    uint64_t empty[kStages];              // each CTA: the leader's MMA commit
    uint64_t tmem_full;                   // each CTA: the leader's commit after a tile
    uint64_t tmem_empty;                  // used in the leader: 2 x kEpiWarps arrivals
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    GroupTable table;
};

// An output tile: its group, its row and column tile inside the group, and its K atoms (128
// elements each).
struct Tile {
    int e, mt, nt, atoms;
};

template <bool kWgrad>
__device__ __forceinline__ int tile_count(const GroupedGemmArgs& g, const GroupTable& t) {
    return kWgrad ? g.groups * g.tiles_m * g.tiles_n : t.tiles2[g.groups] * g.tiles_n;
}

template <bool kWgrad>
__device__ __forceinline__ Tile tile_at(int i, const GroupedGemmArgs& g, const GroupTable& t) {
    Tile r;
    if (kWgrad) {
        const int per = g.tiles_m * g.tiles_n;
        r.e = i / per;
        const int in = i - r.e * per;
        r.nt = in / g.tiles_m;
        r.mt = in - r.nt * g.tiles_m;
        r.atoms = t.tiles[r.e + 1] - t.tiles[r.e];
    } else {
        r.e = find_group(t.tiles2, g.groups, i / g.tiles_n);
        const int rows2 = t.tiles2[r.e + 1] - t.tiles2[r.e];
        const int in = i - t.tiles2[r.e] * g.tiles_n;
        r.nt = in / rows2;
        r.mt = in - r.nt * rows2;
        r.atoms = g.atoms;
    }
    return r;
}

// This warp's 32 rows x 128 columns of the accumulator as output words: 64 of bf16 pairs, 128
// of fp32.  For bf16 the first half is converted while the second is read, so that no more
// than 64 fp32 values are live.
template <bool kF32>
__device__ __forceinline__ void read_accumulator(uint32_t taddr, uint32_t (&w)[kF32 ? 128 : 64]) {
    uint32_t v0[32], v1[32];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        tc_ld_32x32b_x32(taddr + 64 * half, v0);
        tc_ld_32x32b_x32(taddr + 64 * half + 32, v1);
        tc_wait_ld();
        if (kF32) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                w[(kF32 ? 64 : 0) * half + i] = v0[i];
                w[(kF32 ? 64 : 0) * half + (kF32 ? 32 : 0) + i] = v1[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                w[32 * half + i] = pack_bf16x2(v0[2 * i], v0[2 * i + 1]);
                w[32 * half + 16 + i] = pack_bf16x2(v1[2 * i], v1[2 * i + 1]);
            }
            // the first half's pairs exist before the second half is read
            if (half == 0) {
#pragma unroll
                for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(w[i]));
            }
        }
    }
}

template <bool kWgrad, bool kF32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ GroupedGemmArgs g) {
    extern __shared__ uint8_t smem_raw[];
    GroupedSmem& sm = *reinterpret_cast<GroupedSmem*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    const int rank = static_cast<int>(cluster_cta_rank());
    const bool leader = rank == 0;
    const int cluster = blockIdx.x >> 1;
    const int nclusters = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        mbar_init(smem_addr(&sm.tmem_full), 1);
        mbar_init(smem_addr(&sm.tmem_empty), 2 * kEpiWarps);
        mbar_init(smem_addr(&sm.drain), 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_addr(&sm.tmem_base), kTmemCols);
        tmem_relinquish_pair();
    }
    grid_wait_prerequisites();
    grid_launch_dependents();
    if (warp == 2) build_group_table(sm.table, g.offsets, g.groups, g.rows, g.err);
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers exist before anything signals across
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    const int num_tiles = tile_count<kWgrad>(g, sm.table);

    if (warp == 0) {
        // ------------------------------------------------------------------ producer
        if (lane == 0) {
            prefetch_tensormap(&g.amap);
            prefetch_tensormap(&g.bmap);
            prefetch_tensormap(&g.sfamap);
            prefetch_tensormap(&g.sfbmap);
            const uint64_t pol = l2_policy_evict_last();
            int it = 0;
            bool ok = true;
            for (int i = cluster; i < num_tiles && ok; i += nclusters) {
                const Tile t = tile_at<kWgrad>(i, g, sm.table);
                const int p128 = sm.table.tiles[t.e];
                // element coordinates in bytes, scale coordinates in 8-byte units (64 an atom)
                const int a_x = kWgrad ? p128 * 64 : 0, sfa_x = kWgrad ? p128 * 64 : 0;
                const int a_y = (kWgrad ? 0 : sm.table.start[t.e]) + t.mt * 256 + rank * 128;
                const int sfa_y = (kWgrad ? 0 : p128) + 2 * t.mt + rank;
                const int b_x = kWgrad ? p128 * 64 : t.e * g.b_step_atoms * 64;
                const int b_y = t.e * g.b_step_rows + t.nt * 256 + rank * 128;
                const int sfb_y = t.e * g.b_step_groups + 2 * t.nt;
                const int steps = (t.atoms + 1) >> 1;
                for (int ks = 0; ks < steps; ++ks, ++it) {
                    const int s = it % kStages;
                    const uint32_t ph = (it / kStages) & 1;
                    if (!mbar_wait(smem_addr(&sm.empty[s]), ph ^ 1, g.err, kErrGemmProducer, &sm.abort)) {
                        ok = false;
                        break;
                    }
                    if (leader) mbar_arrive_expect_tx(smem_addr(&sm.full[s]), 2 * kStageBytes);
                    const uint32_t bar = cluster_map(smem_addr(&sm.full[s]), 0);
                    tma_load_2d_pair(smem_addr(sm.a[s]), &g.amap, a_x + ks * BKB, a_y, bar, pol);
                    tma_load_2d_pair(smem_addr(sm.b[s]), &g.bmap, b_x + ks * BKB, b_y, bar, pol);
                    tma_load_2d_pair(smem_addr(sm.sfa[s]), &g.sfamap, sfa_x + ks * 128, sfa_y, bar, pol);
                    tma_load_2d_pair(smem_addr(sm.sfb[s]), &g.sfbmap, b_x + ks * 128, sfb_y, bar, pol);
                }
            }
            // Drain (leader): every armed stage, both CTAs' bytes, has landed.
            if (leader) {
                const int armed = it < kStages ? it : kStages;
                for (int i = 1; i <= armed; ++i) {
                    const int j = it - i;
                    mbar_wait_quiet(smem_addr(&sm.full[j % kStages]), (j / kStages) & 1, kWaitLimitNs);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------------ MMA issuer
        // Shared memory is read only between tiles, where the accumulator is awaited anyway (a
        // shared read with MMAs in flight holds this warp until they are done).
        if (leader) {
            int it = 0;
            bool ok = true;
            for (int i = cluster; i < num_tiles && ok; i += nclusters) {
                const int atoms = kWgrad ? tile_at<kWgrad>(i, g, sm.table).atoms : g.atoms;
                const int steps = (atoms + 1) >> 1;
                for (int ks = 0; ks < steps; ++ks, ++it) {
                    if (!named_barrier_and(kBarHandoff, 64, true)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        tc_fence_after_sync();
                        const int s = it % kStages;
                        const int natoms = min(2, atoms - 2 * ks);
                        const uint32_t sf = tmem + kSfTmemBase + s * kSfTmemPerStage;
                        const uint32_t sfa_s = smem_addr(sm.sfa[s]);
                        const uint32_t sfb_s = smem_addr(sm.sfb[s]);
                        const uint64_t adesc = smem_desc(smem_addr(sm.a[s]), 16, 1024, 2);
                        const uint64_t bdesc = smem_desc(smem_addr(sm.b[s]), 16, 1024, 2);
                        for (int a = 0; a < natoms; ++a) {
                            tc_cp_32x128b_warpx4_pair(sf + a * 4, smem_desc(sfa_s + a * 512, 0, 128, 0));
#pragma unroll
                            for (int gb = 0; gb < 2; ++gb)
                                tc_cp_32x128b_warpx4_pair(sf + 8 + (a * 2 + gb) * 4,
                                                          smem_desc(sfb_s + gb * 1024 + a * 512, 0, 128, 0));
#pragma unroll
                            for (int jj = 0; jj < 2; ++jj) {
                                const int j = 2 * a + jj;
                                tc_mma_mxf4_pair(tmem, adesc + 2 * j, bdesc + 2 * j, pair_idesc(jj * 2, 256), sf + a * 4,
                                                 sf + 8 + a * 8, (ks | j) != 0);
                            }
                        }
                        tc_commit_pair_multicast(smem_addr(&sm.empty[s]), 3);
                        if (ks == steps - 1) tc_commit_pair_multicast(smem_addr(&sm.tmem_full), 3);
                    }
                }
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
            bool ok = true;
            for (int i = cluster; i < num_tiles && ok; i += nclusters) {
                const int atoms = kWgrad ? tile_at<kWgrad>(i, g, sm.table).atoms : g.atoms;
                const int steps = (atoms + 1) >> 1;
                for (int ks = 0; ks < steps; ++ks, ++it) {
                    int w = 1;
                    if (lane == 0) {
                        if (ks == 0 && tl > 0)
                            w = mbar_wait(smem_addr(&sm.tmem_empty), (tl - 1) & 1, g.err, kErrGemmMma, &sm.abort);
                        if (w)
                            w = mbar_wait(smem_addr(&sm.full[it % kStages]), (it / kStages) & 1, g.err, kErrGemmMma,
                                          &sm.abort);
                    }
                    if (!named_barrier_and(kBarHandoff, 64, __shfl_sync(0xFFFFFFFFu, w, 0) != 0)) {
                        ok = false;
                        break;
                    }
                }
                tl += steps > 0;
            }
        }
    } else {
        // ------------------------------------------------------------------ epilogue
        const int q = warp & 3;
        const int h = (warp - kEpi0) >> 2;
        const uint32_t obuf = smem_addr(sm.out[warp - kEpi0]);
        const uint64_t pol = l2_policy_evict_first();
        const uint32_t leader_tmem_empty = cluster_map(smem_addr(&sm.tmem_empty), 0);
        if (lane == 0 && g.c_tma) prefetch_tensormap(&g.cmap);
        constexpr int kPer = kF32 ? 16 : 32;   // columns of a 64-byte piece
        constexpr int kPieces = 128 / kPer;
        int tl = 0;
        for (int i = cluster; i < num_tiles; i += nclusters) {
            const Tile t = tile_at<kWgrad>(i, g, sm.table);
            uint32_t w[kF32 ? 128 : 64];
            if (t.atoms > 0) {
                int okw = 1;
                if (warp == kEpi0 && lane == 0)
                    okw = mbar_wait(smem_addr(&sm.tmem_full), tl & 1, g.err, kErrGemmEpilogue, &sm.abort);
                if (!named_barrier_and(kBarEpilogue, kEpiWarps * 32, __shfl_sync(0xFFFFFFFFu, okw, 0) != 0)) break;
                ++tl;
                tc_fence_after_sync();
                read_accumulator<kF32>(tmem + (static_cast<uint32_t>(q * 32) << 16) + h * 128, w);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(leader_tmem_empty);
            } else {
#pragma unroll
                for (int j = 0; j < (kF32 ? 128 : 64); ++j) w[j] = 0u;
            }
            const int64_t base = kWgrad ? static_cast<int64_t>(t.e) * g.m_rows : sm.table.start[t.e];
            const int64_t end = kWgrad ? base + g.m_rows : sm.table.start[t.e + 1];
            const int64_t row0 = base + t.mt * 256 + rank * 128 + q * 32;
            const int64_t col0 = static_cast<int64_t>(t.nt) * 256 + h * 128;
            if (row0 >= end || col0 >= g.n_cols) continue;
            if (g.c_tma && row0 + 32 <= end) {
#pragma unroll
                for (int c = 0; c < kPieces; ++c) {
                    if (col0 + c * kPer >= g.n_cols) break;
                    if (lane == 0) bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(obuf + swz64(lane, j), w[16 * c + 4 * j], w[16 * c + 4 * j + 1], w[16 * c + 4 * j + 2],
                               w[16 * c + 4 * j + 3]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d_hint(&g.cmap, static_cast<int32_t>(col0 + c * kPer), static_cast<int32_t>(row0), obuf,
                                          pol);
                        bulk_commit_group();
                    }
                }
                continue;
            }
            // the group's last rows, or a pitch that no tensor store takes: each lane its row
            const int64_t row = row0 + lane;
            if (row >= end) continue;
            uint32_t* const dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(g.c) + (row * g.ldc + col0) * (kF32 ? 4 : 2));
            const int cols = static_cast<int>(min(g.n_cols - col0, int64_t{128}));
            if (g.c_tma) {
#pragma unroll
                for (int j = 0; j < (kF32 ? 32 : 16); ++j)
                    if ((j + 1) * (kPer / 4) <= cols)
                        reinterpret_cast<uint4*>(dst)[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                if (cols % (kPer / 4) == 0) continue;
            }
            const int from = g.c_tma ? cols / (kPer / 4) * (kPer / 4) : 0;
            if (kF32) {
#pragma unroll
                for (int j = 0; j < (kF32 ? 128 : 64); ++j)
                    if (j >= from && j < cols) dst[j] = w[j];
            } else {
#pragma unroll
                for (int j = 0; j < 128; ++j)
                    if (j >= from && j < cols)
                        reinterpret_cast<uint16_t*>(dst)[j] = static_cast<uint16_t>(w[(j >> 1) & (kF32 ? 127 : 63)] >> (16 * (j & 1)));
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

size_t smem_bytes() { return sizeof(GroupedSmem) + 1024; }

}  // namespace

int gemm_grouped_max_clusters() {
    static int cached[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (cached[dev] > 0) return cached[dev];
    auto kernel = gemm_grouped_kernel<true, true>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes()) != cudaSuccess)
        return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes();
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    cached[dev] = n;
    return n;
}

cudaError_t launch_gemm_grouped(const GroupedGemmArgs& a, bool wgrad, int clusters, cudaStream_t stream) {
    auto kernel = wgrad ? (a.out_f32 ? gemm_grouped_kernel<true, true> : gemm_grouped_kernel<true, false>)
                        : (a.out_f32 ? gemm_grouped_kernel<false, true> : gemm_grouped_kernel<false, false>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes());
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * clusters, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem_bytes();
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mxfp4
