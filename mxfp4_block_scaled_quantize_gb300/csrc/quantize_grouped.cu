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
//   both blobs   a 128 x 128 tile of one group a step, as in the plain quantizer, but the rows
//                of a tile come from anywhere in X, so 256 threads fetch them with 16-byte
//                cp.async (a row of the tile is 256 contiguous bytes) into a ring of three
//                stages, two tiles ahead; each CTA walks a contiguous run of tiles along K, so
//                the index and the group are looked up once a row tile.
//   row blob     no shared memory: a thread takes one block, a warp 32 blocks of one row, so a
//                single token's row is spread over as many warps as it has 1024-element pieces.
#include <cuda_bf16.h>

#include "group_table.cuh"
#include "launch.h"
#include "mx_encode.cuh"
#include "ptx.cuh"
#include "quant_tile.cuh"

namespace mxfp4 {
namespace {

constexpr int kStages = 3;
constexpr int kThreads = 256;
constexpr int kRowThreads = 128;

struct DualSmem {
    uint8_t tile[kStages][kQTileBytes];
    GroupTable table;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// X's row of row i of G, or -1 (recorded) where the index points outside X: such a row is zero.
__device__ __forceinline__ int source_row(const GroupedQuantArgs& p, int i) {
    if (p.row_index == nullptr) return i;
    const int r = __ldg(p.row_index + i);
    if (r >= 0 && r < p.x_rows) return r;
    atomicOr(p.err, kErrGroups);
    return -1;
}

__global__ void __launch_bounds__(kThreads, 2) quantize_grouped_kernel(const GroupedQuantArgs p) {
    extern __shared__ uint8_t smem_raw[];
    DualSmem& sm = *reinterpret_cast<DualSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const uint32_t lane = lane_id();
    grid_wait_prerequisites();
    grid_launch_dependents();
    if (warp == 0) build_group_table(sm.table, p.offsets, p.groups, p.rows, p.err);
    __syncthreads();
    const int64_t total = static_cast<int64_t>(sm.table.tiles[p.groups]) * p.tiles_k;
    const int64_t t0 = total * blockIdx.x / gridDim.x, t1 = total * (blockIdx.x + 1) / gridDim.x;

    // Loader: thread t brings 16-byte chunk t % 16 of rows t / 16 + 16 i of each tile.
    const int lj = tid & 15, lr = tid >> 4;
    int load_gt = -1;
    int src[8];
    auto issue = [&](int64_t t) {
        if (t < t1) {
            const int gt = static_cast<int>(t / p.tiles_k), tk = static_cast<int>(t - static_cast<int64_t>(gt) * p.tiles_k);
            if (gt != load_gt) {
                load_gt = gt;
                const int e = find_group(sm.table.tiles, p.groups, gt);
                const int row0 = sm.table.start[e] + (gt - sm.table.tiles[e]) * kQT;
                const int end = sm.table.start[e + 1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = row0 + lr + 16 * i;
                    src[i] = row < end ? source_row(p, row) : -1;
                }
            }
            const int64_t col = static_cast<int64_t>(tk) * kQT + 8 * lj;
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

    int gt = -1, row0 = 0, live = 0;
    for (int64_t t = t0; t < t1; ++t) {
        cp_async_wait<1>();
        __syncthreads();   // tile t has landed, and every thread is done with tile t - 1
        issue(t + 2);
        const int g = static_cast<int>(t / p.tiles_k), tk = static_cast<int>(t - static_cast<int64_t>(g) * p.tiles_k);
        if (g != gt) {
            gt = g;
            const int e = find_group(sm.table.tiles, p.groups, gt);
            row0 = sm.table.start[e] + (gt - sm.table.tiles[e]) * kQT;
            live = min(sm.table.start[e + 1] - row0, kQT);
        }
        const uint32_t tile = smem_addr(sm.tile[(t - t0) % kStages]);
        const int64_t k0 = static_cast<int64_t>(tk) * kQT;
        uint8_t* const atom_row = p.s_row + (static_cast<int64_t>(gt) * p.tiles_k + tk) * 512;
        uint8_t* const atom_col = p.s_col + (static_cast<int64_t>(tk) * p.tiles_r + gt) * 512;

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
                *reinterpret_cast<uint4*>(p.q_row + static_cast<int64_t>(row0 + r) * p.ldq_row + ((k0 + 32 * b) >> 1)) =
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
        const int64_t off = static_cast<int64_t>(gt) * (kQT / 2) + rb * 16;
        if (kc < p.K) *reinterpret_cast<uint4*>(p.q_col + kc * p.ldq_col + off) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
        if (kc + 1 < p.K)
            *reinterpret_cast<uint4*>(p.q_col + (kc + 1) * p.ldq_col + off) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
        const int kl0 = 2 * pc, kl1 = 2 * pc + 1;
        atom_col[(kl0 & 31) * 16 + (kl0 >> 5) * 4 + rb] = static_cast<uint8_t>(kc < p.K ? byte0 : 0u);
        atom_col[(kl1 & 31) * 16 + (kl1 >> 5) * 4 + rb] = static_cast<uint8_t>(kc + 1 < p.K ? byte1 : 0u);
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
    const int64_t units = static_cast<int64_t>(table.start[p.groups] - first) * pieces;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kRowThreads / 32);
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
        const int row = first + static_cast<int>(u / pieces);
        const int kb = static_cast<int>(u % pieces) * 32 + static_cast<int>(lane);
        int src = 0;
        if (lane == 0) src = source_row(p, row);
        src = __shfl_sync(0xFFFFFFFFu, src, 0);
        uint4 v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = make_uint4(0, 0, 0, 0);
        const int64_t k0 = static_cast<int64_t>(kb) * 32;
        if (src >= 0 && k0 < p.K) {
            const uint16_t* const x = p.x + src * p.ldx + k0;
            if (k0 + 32 <= p.K) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = __ldg(reinterpret_cast<const uint4*>(x) + c);
            } else {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t lo = k0 + 2 * i < p.K ? __ldg(x + 2 * i) : 0u;
                    const uint32_t hi = k0 + 2 * i + 1 < p.K ? __ldg(x + 2 * i + 1) : 0u;
                    w[i] = lo | (hi << 16);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
        }
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) m = absmax2(m, absmax2(absmax2(v[c].x, v[c].y), absmax2(v[c].z, v[c].w)));
        m = absmax2(m, m >> 16) & 0x7FFFu;
        const uint32_t byte = scale_byte(m);
        const uint64_t s2 = pack2(inv_scale_bits(byte), inv_scale_bits(byte));
        if (kb < blocks)
            *reinterpret_cast<uint4*>(p.q_row + static_cast<int64_t>(row) * p.ldq_row + kb * 16) =
                make_uint4(encode8(v[0].x, v[0].y, v[0].z, v[0].w, s2), encode8(v[1].x, v[1].y, v[1].z, v[1].w, s2),
                           encode8(v[2].x, v[2].y, v[2].z, v[2].w, s2), encode8(v[3].x, v[3].y, v[3].z, v[3].w, s2));
        // four lanes hold the four consecutive scale bytes of a row in an atom
        uint32_t word = byte << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
        if ((lane & 3) == 0 && kb < blocks) {
            const int e = find_group(table.start, p.groups, row);
            const int in = row - table.start[e];
            const int64_t atom = static_cast<int64_t>(table.tiles[e] + (in >> 7)) * p.tiles_k + (kb >> 2);
            *reinterpret_cast<uint32_t*>(p.s_row + atom * 512 + (in & 31) * 16 + ((in & 127) >> 5) * 4) = word;
        }
    }
}

}  // namespace

cudaError_t launch_quantize_grouped(const GroupedQuantArgs& a, int sms, cudaStream_t stream) {
    const bool dual = a.q_col != nullptr;
    const size_t smem = dual ? sizeof(DualSmem) + 1024 : 0;
    auto kernel = dual ? quantize_grouped_kernel : quantize_grouped_row_kernel;
    if (dual) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // dual: two CTAs fit an SM; row blob: up to 8, no more than there are warps' worth of pieces
    const int64_t most = dual ? static_cast<int64_t>(a.tiles_r) * a.tiles_k
                              : (static_cast<int64_t>(a.rows) * ((4 * a.tiles_k + 31) / 32) + 3) / (kRowThreads / 32);
    const int64_t cap = static_cast<int64_t>(sms) * (dual ? 2 : 8);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(most < cap ? most : cap), 1, 1);
    cfg.blockDim = dim3(dual ? kThreads : kRowThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mxfp4
