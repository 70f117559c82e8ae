// quantize_grouped.cu -- the MXFP4 quantizer of a grouped linear: rows of bf16 X, gathered by
// an index, cut into groups whose sizes only the device knows.
//
// What it computes.  G[i] = X[index[i]] (or X[i]), i < rows; group e holds rows
// start[e] .. start[e+1].  Row blob: G's rows in blocks of 32 along K, as the plain quantizer's.
// Col blob: for the products that sum over a group's rows, every group's rows are padded to a
// multiple of 128 with zeros, and the columns of that padded matrix are quantized in blocks of
// 32 along it; the padding keeps every block, scale atom and K step inside one group.  The MX
// arithmetic is the plain quantizer's (mx_encode.cuh, quant_tile.cuh).
//
// Both kernels are bound by memory: 2 bytes read and 0.53 (row) or 1.06 (both blobs) written an
// element.
//   both blobs   a 128 x 128 tile of one group a step, in the plain quantizer's way, in one of
//                two kernels.  Rows of X as they are: a producer thread brings tiles as two boxes
//                of a tensor map into a ring of three stages (184 M elements 98 us, 0.86 of the
//                measured copy rate).  Gathered rows come from anywhere in X: every thread
//                fetches its share of a tile two ahead with 16-byte cp.async.  (50 M elements
//                gathered from 4096 rows: gathering tensor copies, four rows each, took 71 us, cp.async
//                from two producer warps 92 us, this 43.)
//   row blob     no shared memory: a warp takes a 1024-element piece of one row, so that a
//                single token's row is spread over as many warps as it has pieces; its loads and
//                stores are whole lines (a lane holding a whole block read 16 bytes of each of 32
//                lines: 26 us for 50 M elements against 22, cold); the next piece is fetched while
//                one is encoded.  A piece that K ends inside is loaded element by element, one after
//                the other: 50 M elements back to back take 15 us at K = 2048, 35 at 2880, 44 at
//                1536, 48 at 1408 and 99 at 512.
#include <cuda_bf16.h>

#include "group_table.cuh"
#include "launch.h"
#include "mx_encode.cuh"
#include "pair_common.cuh"
#include "ptx.cuh"
#include "quant_tile.cuh"

namespace mxfp4 {
namespace {

constexpr int kStages = 3;
constexpr int kWarps = 8;                         // that quantize
constexpr int kThreads = (kWarps + 1) * 32;       // + the producer
constexpr int kGatherThreads = kWarps * 32;       // no producer: each thread fetches its share
constexpr int kRowThreads = 128;
constexpr int kSharedTilesPerCta = 12;            // most tiles a CTA of a launch that two tensors share

// A 128 x 128 tile of a task.
struct Tile {
    int32_t task;   // of the launch
    int32_t gt;     // padded row / 128
    int32_t tk;     // column / 128
    int32_t row0;   // row of G
    int32_t live;   // rows of the tile inside its group
};

struct TileSmem {
    uint8_t tile[kStages][kQTileBytes];
    Tile at[kStages];
    uint64_t full[kStages];
    uint64_t empty[kStages];   // the quantizing warps
    int abort;
    GroupTable table;
};

struct GatherSmem {
    uint8_t tile[kStages][kQTileBytes];
    GroupTable table;
};

// X's row of row i of G, or -1 (recorded) where the index points outside X: such a row is zero.
__device__ __forceinline__ int source_row(const GroupedQuantArgs& p, int i) {
    if (p.row_index == nullptr) return i;
    const int r = __ldg(p.row_index + i);
    if (r >= 0 && r < p.x_rows) return r;
    atomicOr(p.err, kErrGroups);
    return -1;
}

// Padded row tile gt of a task: its group by the table, or by division for equal groups.
__device__ __forceinline__ void place_rows(const GroupedQuantArgs& p, const GroupTable& table, int gt, int* row0, int* live) {
    if (p.offsets == nullptr) {
        int j;
        const int m = p.rows / p.groups, e = small_div(gt, (m + kQT - 1) / kQT, &j);
        *row0 = e * m + j * kQT;
        *live = min(m - j * kQT, kQT);
    } else {
        const int e = find_group(table.tiles, p.groups, gt);
        *row0 = table.start[e] + (gt - table.tiles[e]) * kQT;
        *live = min(table.start[e + 1] - *row0, kQT);
    }
}

__device__ __forceinline__ int row_tiles(const GroupedQuantArgs& p, const GroupTable& table) {
    return p.offsets != nullptr ? table.tiles[p.groups] : p.tiles_r;
}

// One warp's share of the tile in shared memory, both packings.  kMask: rows past t.live hold
// something else than zero.
template <bool kMask>
__device__ __forceinline__ void quantize_tile(const GroupedQuantArgs& p, const Tile& t, uint32_t tile, int warp,
                                              uint32_t lane) {
    const int64_t k0 = static_cast<int64_t>(t.tk) * kQT;
    uint8_t* const atom_row = p.s_row + (static_cast<int64_t>(t.gt) * p.tiles_k + t.tk) * 512;
    uint8_t* const atom_col = p.s_col + (static_cast<int64_t>(t.tk) * p.tiles_r + t.gt) * 512;
    const int live = t.live;

    // rowwise: thread and block mapping of the plain quantizer's rowwise pass
    const int L = 4 * warp + (lane & 3), Q = lane >> 3, r = Q * 32 + L;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int b = ((lane >> 2) & 1) + 2 * i;
        const uint32_t box = tile + (b >> 1) * kQBoxBytes;
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = lds128(box + swz(r, (b & 1) * 4 + c));
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) m = absmax2(m, absmax2(absmax2(v[c].x, v[c].y), absmax2(v[c].z, v[c].w)));
        m = absmax2(m, m >> 16) & 0x7FFFu;
        const uint32_t byte = scale_byte(m);
        const uint64_t s2 = pack2(inv_scale_bits(byte), inv_scale_bits(byte));
        if (r < live)
            *reinterpret_cast<uint4*>(p.q_row + static_cast<int64_t>(t.row0 + r) * p.ldq_row + ((k0 + 32 * b) >> 1)) =
                make_uint4(encode8(v[0].x, v[0].y, v[0].z, v[0].w, s2), encode8(v[1].x, v[1].y, v[1].z, v[1].w, s2),
                           encode8(v[2].x, v[2].y, v[2].z, v[2].w, s2), encode8(v[3].x, v[3].y, v[3].z, v[3].w, s2));
        atom_row[L * 16 + Q * 4 + b] = static_cast<uint8_t>(r < live ? byte : 0u);
    }

    // columnwise: as the plain quantizer's (row block rb walks its rows in the order i ^ 2 rb)
    const int pc = 8 * warp + (lane & 7), rb = lane >> 3;
    const uint32_t box = tile + (pc >> 5) * kQBoxBytes + rb * 32 * 128 + (pc & 3) * 4;
    const int jc = (pc & 31) >> 2;
    uint32_t toff[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int rr = k ^ (2 * rb);
        toff[k] = box + rr * 128 + ((jc ^ rr) << 4);
    }
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = lds32(toff[i & 7] + (i & ~7) * 128);
    if (kMask && live < kQT) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (rb * 32 + (i & ~7) + ((i & 7) ^ (2 * rb)) >= live) w[i] = 0u;
    }
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) m = absmax2(m, w[i]);
    const uint32_t byte0 = scale_byte(m), byte1 = scale_byte(m >> 16);
    const uint64_t s2 = pack2(inv_scale_bits(byte0), inv_scale_bits(byte1));
    const uint32_t sel = 0x3210u ^ (0x1111u * static_cast<uint32_t>(rb));
    uint32_t q0[4], q1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        encode_cols8(&w[8 * j], s2, &q0[j], &q1[j]);
        q0[j] = __byte_perm(q0[j], 0, sel);
        q1[j] = __byte_perm(q1[j], 0, sel);
    }
    const int64_t kc = k0 + 2 * pc;
    const int64_t off = static_cast<int64_t>(t.gt) * (kQT / 2) + rb * 16;
    if (kc < p.K) *reinterpret_cast<uint4*>(p.q_col + kc * p.ldq_col + off) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
    if (kc + 1 < p.K)
        *reinterpret_cast<uint4*>(p.q_col + (kc + 1) * p.ldq_col + off) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
    const int kl0 = 2 * pc, kl1 = 2 * pc + 1;
    atom_col[(kl0 & 31) * 16 + (kl0 >> 5) * 4 + rb] = static_cast<uint8_t>(kc < p.K ? byte0 : 0u);
    atom_col[(kl1 & 31) * 16 + (kl1 >> 5) * 4 + rb] = static_cast<uint8_t>(kc + 1 < p.K ? byte1 : 0u);
}

// The tile t of a launch: its task and place.  at: that of an earlier tile, or task -1; returns
// whether the rows are the same.
__device__ __forceinline__ bool locate(const GroupedQuantBatch& P, const GroupTable& table, int end0, int t, Tile& at) {
    const int j = t < end0 ? 0 : 1;
    const GroupedQuantArgs& p = P.task[j];
    int tk;
    const int gt = small_div(t - (j > 0 ? end0 : 0), p.tiles_k, &tk);
    const bool same = at.task == j && at.gt == gt;
    if (!same) place_rows(p, table, gt, &at.row0, &at.live);
    at.task = j;
    at.gt = gt;
    at.tk = tk;
    return same;
}

// The group table of a launch (one warp), and the tiles of its first task and of all.
__device__ __forceinline__ void build_table(const GroupedQuantBatch& P, GroupTable& table) {
    for (int j = 0; j < P.count; ++j)   // at most one task has offsets
        if (P.task[j].offsets != nullptr)
            build_group_table(table, P.task[j].offsets, P.task[j].groups, P.task[j].rows, P.task[j].err);
}

__device__ __forceinline__ int count_tiles(const GroupedQuantBatch& P, const GroupTable& table, int* end0) {
    *end0 = row_tiles(P.task[0], table) * P.task[0].tiles_k;
    return *end0 + (P.count > 1 ? row_tiles(P.task[1], table) * P.task[1].tiles_k : 0);
}

// Rows of X as they are.
__global__ void __launch_bounds__(kThreads, 2) quantize_grouped_kernel(const __grid_constant__ GroupedQuantBatch P) {
    extern __shared__ uint8_t smem_raw[];
    TileSmem& sm = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    uint32_t* const err = P.task[0].err;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), kWarps);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    grid_wait_prerequisites();
    grid_launch_dependents();
    if (warp == 1) build_table(P, sm.table);
    __syncthreads();
    int end0;
    const int total = count_tiles(P, sm.table, &end0);

    if (warp == kWarps) {
        // ------------------------------------------------------------- producer
        int it = 0;
        Tile at{-1, 0, 0, 0, 0};
        for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
            const int s = it % kStages;
            locate(P, sm.table, end0, t, at);
            int ok = 0;
            if (lane == 0)
                ok = mbar_wait(smem_addr(&sm.empty[s]), ((it / kStages) & 1) ^ 1, err, kErrQuantProducer, &sm.abort) ? 1 : 0;
            if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
            if (lane == 0) {
                const uint32_t bar = smem_addr(&sm.full[s]);
                sm.at[s] = at;
                mbar_arrive_expect_tx(bar, kQTileBytes);
                tma_load_2d(smem_addr(sm.tile[s]), &P.map[at.task], at.tk * kQT, at.row0, bar);
                tma_load_2d(smem_addr(sm.tile[s]) + kQBoxBytes, &P.map[at.task], at.tk * kQT + 64, at.row0, bar);
            }
        }
        // Drain: every armed stage's copies have landed before this warp may leave.
        if (lane == 0) {
            const int armed = it < kStages ? it : kStages;
            for (int i = 1; i <= armed; ++i) {
                const int j = it - i;
                mbar_wait_quiet(smem_addr(&sm.full[j % kStages]), (j / kStages) & 1, kWaitLimitNs);
            }
        }
        return;
    }
    int it = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++it) {
        const int s = it % kStages;
        int ok = 0;
        if (lane == 0)
            ok = mbar_wait(smem_addr(&sm.full[s]), (it / kStages) & 1, err, kErrQuantConsumer, &sm.abort) ? 1 : 0;
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
        const Tile at = sm.at[s];
        // what the boxes hold past the group's end is the next group's
        quantize_tile<true>(P.task[at.task], at, smem_addr(sm.tile[s]), warp, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sm.empty[s]));   // this warp is done with the stage
    }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// One or two tasks with gathered rows.  CTA b takes the tiles of a contiguous run, along K first, so
// that a row tile's group and its source rows are looked up once.
__global__ void __launch_bounds__(kGatherThreads, 2)
    quantize_grouped_gather_kernel(const __grid_constant__ GroupedQuantBatch P) {
    extern __shared__ uint8_t smem_raw[];
    GatherSmem& sm = *reinterpret_cast<GatherSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                    ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    grid_wait_prerequisites();
    grid_launch_dependents();
    if (warp == 0) build_table(P, sm.table);
    __syncthreads();
    int end0;
    const int total = count_tiles(P, sm.table, &end0);
    const int t0 = static_cast<int>(static_cast<int64_t>(total) * blockIdx.x / gridDim.x);
    const int t1 = static_cast<int>(static_cast<int64_t>(total) * (blockIdx.x + 1) / gridDim.x);
    // Loader: thread t brings 16-byte chunk t % 16 of rows t / 16 + 16 i of each tile; rows past
    // the group's end and rows from outside X arrive as zeros.
    const int lj = tid & 15, lr = tid >> 4;
    Tile load_at{-1, 0, 0, 0, 0};
    int src[8];
    auto issue = [&](int t) {
        if (t < t1) {
            const bool same = locate(P, sm.table, end0, t, load_at);
            const GroupedQuantArgs& p = P.task[load_at.task];
            if (!same) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = lr + 16 * i;
                    src[i] = r < load_at.live ? source_row(p, load_at.row0 + r) : -1;
                }
            }
            const int64_t col = static_cast<int64_t>(load_at.tk) * kQT + 8 * lj;
            const uint32_t bytes = col >= p.K ? 0u : static_cast<uint32_t>(min(p.K - col, int64_t{8})) * 2u;
            const uint32_t box = smem_addr(sm.tile[(t - t0) % kStages]) + (lj >> 3) * kQBoxBytes;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool some = src[i] >= 0 && bytes != 0;
                cp_async16(box + swz(lr + 16 * i, lj & 7), some ? p.x + src[i] * p.ldx + col : p.x, some ? bytes : 0u);
            }
        }
        cp_async_commit();
    };
    issue(t0);
    issue(t0 + 1);
    Tile at{-1, 0, 0, 0, 0};
    for (int t = t0; t < t1; ++t) {
        cp_async_wait<1>();
        __syncthreads();   // tile t has landed, and every thread is done with tile t - 1
        issue(t + 2);
        locate(P, sm.table, end0, t, at);
        quantize_tile<false>(P.task[at.task], at, smem_addr(sm.tile[(t - t0) % kStages]), warp, lane);
    }
}

__global__ void __launch_bounds__(kRowThreads) quantize_grouped_row_kernel(const GroupedQuantArgs p) {
    __shared__ GroupTable table;
    const uint32_t lane = lane_id();
    grid_wait_prerequisites();
    grid_launch_dependents();
    if (threadIdx.x < 32) build_group_table(table, p.offsets, p.groups, p.rows, p.err);
    __syncthreads();
    const int blocks = 4 * p.tiles_k;                 // 32-element blocks of a row
    const int pieces = (blocks + 31) >> 5;
    const int first = table.start[0];
    // a warp's run of pieces: consecutive, so rows and pieces are counted up
    const int64_t units = static_cast<int64_t>(table.start[p.groups] - first) * pieces;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
    const int64_t me = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
    const int64_t u0 = units * me / warps;
    int n = static_cast<int>(units * (me + 1) / warps - u0);
    if (n == 0) return;
    int row = first + static_cast<int>(u0 / pieces), piece = static_cast<int>(u0 % pieces);
    int e = find_group(table.start, p.groups, row);
    // the source rows of 32 rows ahead, one a lane
    int ahead = 0, ahead0 = row;
    const int rows_end = table.start[p.groups];
    auto source = [&]() {
        if (p.row_index == nullptr) return row;
        if (row - ahead0 == 32 || row == ahead0) {
            ahead0 = row;
            ahead = row + static_cast<int>(lane) < rows_end ? source_row(p, row + static_cast<int>(lane)) : 0;
        }
        return __shfl_sync(0xFFFFFFFFu, ahead, row - ahead0);
    };
    int src = source();
    int64_t atoms = 0;   // of this row's padded row: first scale atom, and the row inside it
    int in = 0;
    auto place = [&]() {
        while (row >= table.start[e + 1]) ++e;
        in = row - table.start[e];
        atoms = static_cast<int64_t>(table.tiles[e] + (in >> 7)) * p.tiles_k;
    };
    place();
    // Load c of a piece: 8 elements a lane, 256 consecutive ones a warp; four lanes hold a block.
    auto fetch = [&](uint4 (&v)[4]) {
        const int64_t k0 = static_cast<int64_t>(piece) * 1024 + 8 * lane;
        const uint16_t* const x = p.x + src * p.ldx + k0;
        if (src >= 0 && (piece + 1) * int64_t{1024} <= p.K) {   // a whole piece: the usual case
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = __ldg(reinterpret_cast<const uint4*>(x) + 32 * c);
            return;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
            for (int i = 0; i < 8; ++i)
                if (src >= 0 && k0 + 256 * c + i < p.K)
                    w[i >> 1] |= static_cast<uint32_t>(__ldg(x + 256 * c + i)) << (16 * (i & 1));
            v[c] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    };
    uint4 cur[4];
    fetch(cur);
    for (; n > 0; --n) {
        const int kb0 = piece * 32;
        uint8_t* const q_at = p.q_row + static_cast<int64_t>(row) * p.ldq_row + kb0 * 16 + 4 * lane;
        uint8_t* const s_at = p.s_row + atoms * 512 + (in & 31) * 16 + ((in & 127) >> 5) * 4;
        // the next piece's elements are on their way while this one is encoded
        uint4 nxt[4];
        if (n > 1) {
            if (++piece == pieces) {
                piece = 0;
                ++row;
                src = source();
                place();
            }
            fetch(nxt);
        }
        // the blocks' largest magnitudes, two loads to a word: own 8 elements, then the 4 lanes
        uint32_t m[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 a = cur[2 * h], b = cur[2 * h + 1];
            const uint32_t ma = absmax2(absmax2(a.x, a.y), absmax2(a.z, a.w));
            const uint32_t mb = absmax2(absmax2(b.x, b.y), absmax2(b.z, b.w));
            m[h] = absmax2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
            m[h] = absmax2(m[h], __shfl_xor_sync(0xFFFFFFFFu, m[h], 1));
            m[h] = absmax2(m[h], __shfl_xor_sync(0xFFFFFFFFu, m[h], 2));
        }
        uint32_t byte[4], q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            byte[c] = scale_byte(c & 1 ? m[c >> 1] >> 16 : m[c >> 1]);
            const uint32_t inv = inv_scale_bits(byte[c]);
            q[c] = encode8(cur[c].x, cur[c].y, cur[c].z, cur[c].w, pack2(inv, inv));
        }
        // lane l stores the scale byte of its block in load l % 4
        const uint32_t mine = (lane & 2) ? ((lane & 1) ? byte[3] : byte[2]) : ((lane & 1) ? byte[1] : byte[0]);
        const int kb = kb0 + 8 * static_cast<int>(lane & 3) + static_cast<int>(lane >> 2);
        if (kb0 + 32 <= blocks) {
#pragma unroll
            for (int c = 0; c < 4; ++c) *reinterpret_cast<uint32_t*>(q_at + 128 * c) = q[c];
            s_at[(kb >> 2) * 512 + (kb & 3)] = static_cast<uint8_t>(mine);
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (kb0 + 8 * c + static_cast<int>(lane >> 2) < blocks) *reinterpret_cast<uint32_t*>(q_at + 128 * c) = q[c];
            if (kb < blocks) s_at[(kb >> 2) * 512 + (kb & 3)] = static_cast<uint8_t>(mine);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) cur[c] = nxt[c];
    }
}

}  // namespace

namespace {

struct Launch {
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = {};
    Launch(int64_t most, int64_t cap, int threads, size_t smem, cudaStream_t stream) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(static_cast<unsigned>(most < cap ? most : cap), 1, 1);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
};

int64_t tiles_of(const GroupedQuantArgs& a) { return static_cast<int64_t>(a.tiles_r) * a.tiles_k; }

cudaError_t launch_gather(const GroupedQuantBatch& b, int64_t tiles, int sms, cudaStream_t stream) {
    const size_t smem = sizeof(GatherSmem) + 1024;
    const cudaError_t e =
        cudaFuncSetAttribute(quantize_grouped_gather_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const Launch l(tiles, static_cast<int64_t>(sms) * 2, kGatherThreads, smem, stream);
    return cudaLaunchKernelEx(&l.cfg, quantize_grouped_gather_kernel, b);
}

}  // namespace

cudaError_t launch_quantize_grouped(const GroupedQuantBatch& b, int sms, cudaStream_t stream) {
    const bool gather = b.task[0].row_index != nullptr || (b.count > 1 && b.task[1].row_index != nullptr);
    const int64_t tiles = tiles_of(b.task[0]) + (b.count > 1 ? tiles_of(b.task[1]) : 0);
    if (b.count > 1 && gather && tiles > static_cast<int64_t>(sms) * 2 * kSharedTilesPerCta) {
        // Two small tensors share the gathering kernel's launch, larger ones each take the kernel
        // that they need.  A training step as graph replays, shared and apart, in us: 8 groups of 512 x 512 and 1024
        // rows 29.5 and 33.9; 8 of 1536 x 1536, 2048 rows, 60.3 and 64.8; 8 of 2048 x 2048, 8192
        // rows (10 tiles a CTA), 124 and 128; 16 of them, 4096 rows (16 a CTA), 130.7 and 129.8;
        // 64 of 1408 x 2048, 24576 rows, 357 and 348.
        for (int j = 0; j < b.count; ++j) {
            GroupedQuantBatch one = b;
            one.task[0] = b.task[j];
            one.map[0] = b.map[j];
            one.count = 1;
            const cudaError_t e = launch_quantize_grouped(one, sms, stream);
            if (e != cudaSuccess) return e;
        }
        return cudaSuccess;
    }
    const GroupedQuantArgs& a = b.task[0];
    if (a.q_col == nullptr) {
        // up to 8 CTAs an SM, no more than there are pieces for their warps
        const int64_t pieces = static_cast<int64_t>(a.rows) * ((4 * a.tiles_k + 31) / 32);
        const Launch l((pieces + kRowThreads / 32 - 1) / (kRowThreads / 32), static_cast<int64_t>(sms) * 8, kRowThreads, 0,
                       stream);
        return cudaLaunchKernelEx(&l.cfg, quantize_grouped_row_kernel, a);
    }
    if (gather) return launch_gather(b, tiles, sms, stream);
    const size_t smem = sizeof(TileSmem) + 1024;
    const cudaError_t e = cudaFuncSetAttribute(quantize_grouped_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const Launch l(tiles, static_cast<int64_t>(sms) * 2, kThreads, smem, stream);
    return cudaLaunchKernelEx(&l.cfg, quantize_grouped_kernel, b);
}

}  // namespace mxfp4
