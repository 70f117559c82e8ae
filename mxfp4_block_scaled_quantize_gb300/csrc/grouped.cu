// grouped.cu -- host side of the linears grouped by expert (include/mxfp4.h): argument checks,
// tensor maps and launches.  Nothing here reads the group offsets: they stay on the device.
#include <cstring>

#include "launch.h"
#include "mxfp4.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 512;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t pad128(int64_t n) { return cdiv(n, 128) * 128; }
inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

// Most padded rows that `rows` rows in `groups` groups can take, in units of `tile` rows.
int64_t most_tiles(int64_t rows, int64_t groups, bool equal, int64_t tile) {
    if (equal) return groups * cdiv(rows / groups, tile);
    return (rows + (tile - 1) * (groups < rows ? groups : rows)) / tile;
}

bool shape_ok(int64_t rows, int64_t k, int64_t groups, bool equal) {
    if (groups < 1 || groups > MXFP4_MAX_GROUPS || rows < 0 || rows > kMaxDim || k < 1 || k > kMaxDim) return false;
    if (equal && rows % groups != 0) return false;
    return 128 * most_tiles(rows, groups, equal, 128) <= kMaxDim;
}

mxfp4_status gemm_args_ok(mxfp4_grouped_form form, const void* a_q, const void* a_s, const void* b_q, const void* b_s,
                          const int32_t* offsets, int64_t groups, int64_t rows, int64_t N, int64_t K, const void* c,
                          int64_t ldc, mxfp4_out_dtype out_dtype) {
    if (form != MXFP4_GROUPED_FWD && form != MXFP4_GROUPED_DGRAD && form != MXFP4_GROUPED_WGRAD)
        return MXFP4_ERR_INVALID_ARG;
    if (!shape_ok(rows, K, groups, offsets == nullptr) || N < 1 || N > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (pad128(N) * groups > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (out_dtype != MXFP4_OUT_BF16 && out_dtype != MXFP4_OUT_F32) return MXFP4_ERR_INVALID_ARG;
    const int64_t cols = form == MXFP4_GROUPED_FWD ? N : K;
    if (ldc < cols || ldc > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (rows > 0 && (!a_q || !a_s || !b_q || !b_s)) return MXFP4_ERR_INVALID_ARG;
    if ((rows > 0 || form == MXFP4_GROUPED_WGRAD) && c == nullptr) return MXFP4_ERR_INVALID_ARG;
    if (!aligned16(a_q) || !aligned16(a_s) || !aligned16(b_q) || !aligned16(b_s) || !aligned16(c) ||
        !aligned(offsets, 4))
        return MXFP4_ERR_MISALIGNED;
    const int64_t tiles = form == MXFP4_GROUPED_WGRAD ? groups * cdiv(N, 256) * cdiv(K, 256)
                                                      : most_tiles(rows, groups, offsets == nullptr, 256) * cdiv(cols, 256);
    if (tiles > (int64_t{1} << 31) - 1) return MXFP4_ERR_INVALID_ARG;
    return MXFP4_OK;
}

// The elements [rows, packed / 2] of a blob, boxes of 128 rows x 128 bytes, and its scales as
// rows of 128-row atom groups in 8-byte units, boxes of `groups` x 2 atoms.
bool blob_maps(CUtensorMap* q, CUtensorMap* s, const void* qp, const void* sp, int64_t rows, int64_t packed,
               int64_t scale_rows, uint32_t groups) {
    return mxfp4::encode_map_2d(q, CU_TENSOR_MAP_DATA_TYPE_UINT8, qp, static_cast<uint64_t>(packed / 2),
                                static_cast<uint64_t>(rows), static_cast<uint64_t>(packed / 2), 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B) &&
           mxfp4::encode_map_2d(s, CU_TENSOR_MAP_DATA_TYPE_UINT64, sp, static_cast<uint64_t>(packed / 128) * 64,
                                static_cast<uint64_t>(scale_rows / 128), static_cast<uint64_t>(packed / 128) * 512, 128,
                                groups, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace

extern "C" {

mxfp4_status mxfp4_grouped_sizes(int64_t rows, int64_t k, int64_t groups, int32_t equal, size_t* q_row, size_t* s_row,
                                 size_t* q_col, size_t* s_col, int64_t* capacity) {
    if (!shape_ok(rows, k, groups, equal != 0)) return MXFP4_ERR_INVALID_ARG;
    const int64_t cap = 128 * most_tiles(rows, groups, equal != 0, 128), kp = pad128(k);
    if (q_row) *q_row = static_cast<size_t>(rows) * static_cast<size_t>(kp / 2);
    if (s_row) *s_row = static_cast<size_t>(cap) * static_cast<size_t>(kp / 32);
    if (q_col) *q_col = static_cast<size_t>(k) * static_cast<size_t>(cap / 2);
    if (s_col) *s_col = static_cast<size_t>(kp) * static_cast<size_t>(cap / 32);
    if (capacity) *capacity = cap;
    return MXFP4_OK;
}

mxfp4_status mxfp4_quantize_grouped(const void* x, int64_t x_rows, int64_t K, int64_t ldx, const int32_t* row_index,
                                    const int32_t* offsets, int64_t groups, int64_t rows, void* q_row, void* s_row,
                                    void* q_col, void* s_col, mxfp4_stream_t stream) {
    if (!shape_ok(rows, K, groups, offsets == nullptr)) return MXFP4_ERR_INVALID_ARG;
    if (x_rows < 0 || x_rows > kMaxDim || ldx < K || ldx > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (row_index == nullptr && x_rows < rows) return MXFP4_ERR_INVALID_ARG;
    if ((q_col == nullptr) != (s_col == nullptr)) return MXFP4_ERR_INVALID_ARG;
    if (rows > 0 && (!q_row || !s_row || (!x && x_rows > 0))) return MXFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || ldx % 8 != 0 || !aligned16(q_row) || !aligned16(s_row) || !aligned16(q_col) ||
        !aligned16(s_col) || !aligned(row_index, 4) || !aligned(offsets, 4))
        return MXFP4_ERR_MISALIGNED;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK) return static_cast<mxfp4_status>(st);
    if (rows == 0) return MXFP4_OK;
    mxfp4::GroupedQuantArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = static_cast<const uint16_t*>(x);
    a.ldx = ldx;
    a.K = K;
    a.x_rows = static_cast<int32_t>(x_rows);
    a.rows = static_cast<int32_t>(rows);
    a.row_index = row_index;
    a.offsets = offsets;
    a.groups = static_cast<int32_t>(groups);
    a.tiles_k = static_cast<int32_t>(pad128(K) / 128);
    a.tiles_r = static_cast<int32_t>(most_tiles(rows, groups, offsets == nullptr, 128));
    a.q_row = static_cast<uint8_t*>(q_row);
    a.s_row = static_cast<uint8_t*>(s_row);
    a.q_col = static_cast<uint8_t*>(q_col);
    a.s_col = static_cast<uint8_t*>(s_col);
    a.ldq_row = pad128(K) / 2;
    a.ldq_col = static_cast<int64_t>(a.tiles_r) * 64;
    a.err = err;
    return mxfp4::launch_quantize_grouped(a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MXFP4_OK
                                                                                                         : MXFP4_ERR_CUDA;
}

mxfp4_status mxfp4_gemm_grouped(mxfp4_grouped_form form, const void* a_q, const void* a_s, const void* b_q,
                                const void* b_s, const int32_t* offsets, int64_t groups, int64_t rows, int64_t N,
                                int64_t K, void* c, int64_t ldc, mxfp4_out_dtype out_dtype, mxfp4_stream_t stream) {
    const mxfp4_status ok = gemm_args_ok(form, a_q, a_s, b_q, b_s, offsets, groups, rows, N, K, c, ldc, out_dtype);
    if (ok != MXFP4_OK) return ok;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK) return static_cast<mxfp4_status>(st);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool wgrad = form == MXFP4_GROUPED_WGRAD;
    const int64_t esize = out_dtype == MXFP4_OUT_F32 ? 4 : 2;
    if (rows == 0) {
        if (!wgrad) return MXFP4_OK;
        return cudaMemset2DAsync(c, static_cast<size_t>(ldc * esize), 0, static_cast<size_t>(K * esize),
                                 static_cast<size_t>(groups * N), s) == cudaSuccess
                   ? MXFP4_OK
                   : MXFP4_ERR_CUDA;
    }
    mxfp4::GroupedGemmArgs g;
    std::memset(&g, 0, sizeof(g));
    const int64_t cap = 128 * most_tiles(rows, groups, offsets == nullptr, 128);
    const int64_t kp = pad128(K), np = pad128(N);
    bool maps;
    int64_t tiles;
    if (form == MXFP4_GROUPED_FWD) {
        maps = blob_maps(&g.amap, &g.sfamap, a_q, a_s, rows, kp, cap, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, b_q, b_s, groups * N, kp, groups * np, 2);
        g.atoms = static_cast<int32_t>(kp / 128);
        g.b_step_rows = static_cast<int32_t>(N);
        g.b_step_groups = static_cast<int32_t>(np / 128);
        g.n_cols = N;
    } else if (form == MXFP4_GROUPED_DGRAD) {
        maps = blob_maps(&g.amap, &g.sfamap, a_q, a_s, rows, np, cap, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, b_q, b_s, K, groups * np, kp, 2);
        g.atoms = static_cast<int32_t>(np / 128);
        g.b_step_atoms = static_cast<int32_t>(np / 128);
        g.n_cols = K;
    } else {
        maps = blob_maps(&g.amap, &g.sfamap, a_q, a_s, N, cap, np, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, b_q, b_s, K, cap, kp, 2);
        g.tiles_m = static_cast<int32_t>(cdiv(N, 256));
        g.m_rows = N;
        g.n_cols = K;
    }
    if (!maps) return MXFP4_ERR_CUDA;
    g.tiles_n = static_cast<int32_t>(cdiv(g.n_cols, 256));
    tiles = wgrad ? groups * g.tiles_m * g.tiles_n : most_tiles(rows, groups, offsets == nullptr, 256) * g.tiles_n;
    g.c_tma = (ldc * esize) % 16 == 0 &&
              mxfp4::encode_map_2d(&g.cmap, out_dtype == MXFP4_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                                       : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                   c, static_cast<uint64_t>(g.n_cols), static_cast<uint64_t>(wgrad ? groups * N : rows),
                                   static_cast<uint64_t>(ldc * esize), static_cast<uint32_t>(64 / esize), 32,
                                   CU_TENSOR_MAP_SWIZZLE_64B);
    g.offsets = offsets;
    g.groups = static_cast<int32_t>(groups);
    g.rows = static_cast<int32_t>(rows);
    g.c = c;
    g.ldc = ldc;
    g.out_f32 = out_dtype == MXFP4_OUT_F32 ? 1 : 0;
    g.err = err;
    const int most = mxfp4::gemm_grouped_max_clusters();
    if (most <= 0) return MXFP4_ERR_CUDA;
    const int clusters = static_cast<int>(tiles < most ? tiles : most);
    return mxfp4::launch_gemm_grouped(g, wgrad, clusters, s) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

}  // extern "C"
