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

struct Device {
    int sms;
    uint32_t* err;
};

mxfp4_status device(Device* d) { return static_cast<mxfp4_status>(mxfp4::device_info(&d->sms, &d->err)); }

// The arguments of mxfp4_quantize_grouped and of mxfp4_gemm_grouped.
struct Quantize {
    const void* x;
    int64_t x_rows, K, ldx;
    const int32_t* row_index;
    const int32_t* offsets;
    int64_t groups, rows;
    void* blob[4];
};

struct Product {
    mxfp4_grouped_form form;
    const void *a_q, *a_s, *b_q, *b_s;
    const int32_t* offsets;
    int64_t groups, rows, N, K;
    void* c;
    int64_t ldc;
    mxfp4_out_dtype out;
};

mxfp4_status check(const Quantize& t) {
    if (!shape_ok(t.rows, t.K, t.groups, t.offsets == nullptr)) return MXFP4_ERR_INVALID_ARG;
    if (t.x_rows < 0 || t.x_rows > kMaxDim || t.ldx < t.K || t.ldx > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (t.row_index == nullptr && t.x_rows < t.rows) return MXFP4_ERR_INVALID_ARG;
    if ((t.blob[2] == nullptr) != (t.blob[3] == nullptr)) return MXFP4_ERR_INVALID_ARG;
    if (t.rows > 0 && (!t.blob[0] || !t.blob[1] || !t.x || t.x_rows < 1)) return MXFP4_ERR_INVALID_ARG;
    if (!aligned16(t.x) || t.ldx % 8 != 0 || !aligned(t.row_index, 4) || !aligned(t.offsets, 4))
        return MXFP4_ERR_MISALIGNED;
    for (const void* p : t.blob)
        if (!aligned16(p)) return MXFP4_ERR_MISALIGNED;
    // two tensors' tiles are counted in 32 bits
    if (most_tiles(t.rows, t.groups, t.offsets == nullptr, 128) * (pad128(t.K) / 128) > (int64_t{1} << 30) - 1)
        return MXFP4_ERR_INVALID_ARG;
    return MXFP4_OK;
}

mxfp4_status check(const Product& t) {
    if (t.form != MXFP4_GROUPED_FWD && t.form != MXFP4_GROUPED_DGRAD && t.form != MXFP4_GROUPED_WGRAD)
        return MXFP4_ERR_INVALID_ARG;
    if (!shape_ok(t.rows, t.K, t.groups, t.offsets == nullptr) || t.N < 1 || t.N > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (pad128(t.N) * t.groups > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (t.out != MXFP4_OUT_BF16 && t.out != MXFP4_OUT_F32) return MXFP4_ERR_INVALID_ARG;
    const bool wgrad = t.form == MXFP4_GROUPED_WGRAD;
    const int64_t cols = t.form == MXFP4_GROUPED_FWD ? t.N : t.K;
    if (t.ldc < cols || t.ldc > kMaxDim) return MXFP4_ERR_INVALID_ARG;
    if (t.rows > 0 && (!t.a_q || !t.a_s || !t.b_q || !t.b_s)) return MXFP4_ERR_INVALID_ARG;
    if ((t.rows > 0 || wgrad) && t.c == nullptr) return MXFP4_ERR_INVALID_ARG;
    if (!aligned16(t.a_q) || !aligned16(t.a_s) || !aligned16(t.b_q) || !aligned16(t.b_s) || !aligned16(t.c) ||
        !aligned(t.offsets, 4))
        return MXFP4_ERR_MISALIGNED;
    const int64_t tiles = wgrad ? t.groups * cdiv(t.N, 256) * cdiv(t.K, 256)
                                : most_tiles(t.rows, t.groups, t.offsets == nullptr, 256) * cdiv(cols, 256);
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

// Appends a checked tensor with rows to the batch.
mxfp4_status append(const Quantize& t, const Device& dev, mxfp4::GroupedQuantBatch* b) {
    mxfp4::GroupedQuantArgs& a = b->task[b->count];
    a.x = static_cast<const uint16_t*>(t.x);
    a.ldx = t.ldx;
    a.K = t.K;
    a.x_rows = static_cast<int32_t>(t.x_rows);
    a.rows = static_cast<int32_t>(t.rows);
    a.row_index = t.row_index;
    a.offsets = t.offsets;
    a.groups = static_cast<int32_t>(t.groups);
    a.tiles_k = static_cast<int32_t>(pad128(t.K) / 128);
    a.tiles_r = static_cast<int32_t>(most_tiles(t.rows, t.groups, t.offsets == nullptr, 128));
    a.q_row = static_cast<uint8_t*>(t.blob[0]);
    a.s_row = static_cast<uint8_t*>(t.blob[1]);
    a.q_col = static_cast<uint8_t*>(t.blob[2]);
    a.s_col = static_cast<uint8_t*>(t.blob[3]);
    a.ldq_row = pad128(t.K) / 2;
    a.ldq_col = static_cast<int64_t>(a.tiles_r) * 64;
    a.err = dev.err;
    if (t.row_index == nullptr &&
        !mxfp4::encode_map_2d(&b->map[b->count], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t.x, static_cast<uint64_t>(t.K),
                              static_cast<uint64_t>(t.x_rows), static_cast<uint64_t>(t.ldx) * 2, 64, 128,
                              CU_TENSOR_MAP_SWIZZLE_128B))
        return MXFP4_ERR_CUDA;
    ++b->count;
    return MXFP4_OK;
}

// t, and then `also` where it is given and both write both blobs, in one launch; else in two.
mxfp4_status launch(const Quantize& t, const Quantize* also, const Device& dev, cudaStream_t stream) {
    mxfp4::GroupedQuantBatch b;
    std::memset(&b, 0, sizeof(b));
    const bool together = also != nullptr && t.blob[2] != nullptr && also->blob[2] != nullptr;
    mxfp4_status st = append(t, dev, &b);
    if (st == MXFP4_OK && together) st = append(*also, dev, &b);
    if (st != MXFP4_OK) return st;
    if (mxfp4::launch_quantize_grouped(b, dev.sms, stream) != cudaSuccess) return MXFP4_ERR_CUDA;
    return also != nullptr && !together ? launch(*also, nullptr, dev, stream) : MXFP4_OK;
}

mxfp4_status launch(const Product& t, const Device& dev, cudaStream_t stream) {
    const bool wgrad = t.form == MXFP4_GROUPED_WGRAD;
    const int64_t esize = t.out == MXFP4_OUT_F32 ? 4 : 2;
    if (t.rows == 0) {
        if (!wgrad) return MXFP4_OK;
        return cudaMemset2DAsync(t.c, static_cast<size_t>(t.ldc * esize), 0, static_cast<size_t>(t.K * esize),
                                 static_cast<size_t>(t.groups * t.N), stream) == cudaSuccess
                   ? MXFP4_OK
                   : MXFP4_ERR_CUDA;
    }
    mxfp4::GroupedGemmArgs g;
    std::memset(&g, 0, sizeof(g));
    const bool equal = t.offsets == nullptr;
    const int64_t cap = 128 * most_tiles(t.rows, t.groups, equal, 128);
    const int64_t kp = pad128(t.K), np = pad128(t.N);
    bool maps;
    if (t.form == MXFP4_GROUPED_FWD) {
        maps = blob_maps(&g.amap, &g.sfamap, t.a_q, t.a_s, t.rows, kp, cap, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, t.b_q, t.b_s, t.groups * t.N, kp, t.groups * np, 2);
        g.atoms = static_cast<int32_t>(kp / 128);
        g.b_step_rows = static_cast<int32_t>(t.N);
        g.b_step_groups = static_cast<int32_t>(np / 128);
        g.n_cols = t.N;
    } else if (t.form == MXFP4_GROUPED_DGRAD) {
        maps = blob_maps(&g.amap, &g.sfamap, t.a_q, t.a_s, t.rows, np, cap, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, t.b_q, t.b_s, t.K, t.groups * np, kp, 2);
        g.atoms = static_cast<int32_t>(np / 128);
        g.b_step_atoms = static_cast<int32_t>(np / 128);
        g.n_cols = t.K;
    } else {
        maps = blob_maps(&g.amap, &g.sfamap, t.a_q, t.a_s, t.N, cap, np, 1) &&
               blob_maps(&g.bmap, &g.sfbmap, t.b_q, t.b_s, t.K, cap, kp, 2);
        g.tiles_m = static_cast<int32_t>(cdiv(t.N, 256));
        g.m_rows = t.N;
        g.n_cols = t.K;
    }
    if (!maps) return MXFP4_ERR_CUDA;
    g.tiles_n = static_cast<int32_t>(cdiv(g.n_cols, 256));
    const int64_t tiles = wgrad ? t.groups * g.tiles_m * g.tiles_n : most_tiles(t.rows, t.groups, equal, 256) * g.tiles_n;
    g.c_tma = (t.ldc * esize) % 16 == 0 &&
              mxfp4::encode_map_2d(&g.cmap, t.out == MXFP4_OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                   t.c, static_cast<uint64_t>(g.n_cols),
                                   static_cast<uint64_t>(wgrad ? t.groups * t.N : t.rows),
                                   static_cast<uint64_t>(t.ldc * esize), static_cast<uint32_t>(64 / esize), 32,
                                   CU_TENSOR_MAP_SWIZZLE_64B);
    g.offsets = t.offsets;
    g.groups = static_cast<int32_t>(t.groups);
    g.rows = static_cast<int32_t>(t.rows);
    g.c = t.c;
    g.ldc = t.ldc;
    g.out_f32 = t.out == MXFP4_OUT_F32 ? 1 : 0;
    g.err = dev.err;
    const int most = mxfp4::gemm_grouped_max_clusters();
    if (most <= 0) return MXFP4_ERR_CUDA;
    const int clusters = static_cast<int>(tiles < most ? tiles : most);
    return mxfp4::launch_gemm_grouped(g, wgrad, clusters, stream) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
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
    const Quantize t{x, x_rows, K, ldx, row_index, offsets, groups, rows, {q_row, s_row, q_col, s_col}};
    mxfp4_status st = check(t);
    if (st != MXFP4_OK) return st;
    Device dev;
    st = device(&dev);
    if (st != MXFP4_OK || rows == 0) return st;
    return launch(t, nullptr, dev, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_gemm_grouped(mxfp4_grouped_form form, const void* a_q, const void* a_s, const void* b_q,
                                const void* b_s, const int32_t* offsets, int64_t groups, int64_t rows, int64_t N,
                                int64_t K, void* c, int64_t ldc, mxfp4_out_dtype out_dtype, mxfp4_stream_t stream) {
    const Product t{form, a_q, a_s, b_q, b_s, offsets, groups, rows, N, K, c, ldc, out_dtype};
    mxfp4_status st = check(t);
    if (st != MXFP4_OK) return st;
    Device dev;
    st = device(&dev);
    if (st != MXFP4_OK) return st;
    return launch(t, dev, reinterpret_cast<cudaStream_t>(stream));
}

mxfp4_status mxfp4_grouped_forward(const mxfp4_grouped_linear* l, const void* x, int64_t x_rows, int64_t ldx,
                                   const int32_t* row_index, const int32_t* offsets, int64_t rows, const void* w,
                                   mxfp4_stream_t stream) {
    if (l == nullptr || offsets == nullptr) return MXFP4_ERR_INVALID_ARG;
    const int64_t E = l->groups, N = l->N, K = l->K;
    const Quantize qx{x, x_rows, K, ldx, row_index, offsets, E, rows,
                      {l->x_blobs[0], l->x_blobs[1], l->x_blobs[2], l->x_blobs[3]}};
    const Quantize qw{w, E * N, K, K, nullptr, nullptr, E, E * N,
                      {l->w_blobs[0], l->w_blobs[1], l->w_blobs[2], l->w_blobs[3]}};
    const Product y{MXFP4_GROUPED_FWD, l->x_blobs[0], l->x_blobs[1], l->w_blobs[0], l->w_blobs[1], offsets, E, rows, N, K,
                    l->y, N, static_cast<mxfp4_out_dtype>(l->out_dtype)};
    mxfp4_status st = check(y);   // first: it bounds E and N, whose product qw holds
    if (st == MXFP4_OK) st = check(qx);
    if (st == MXFP4_OK && w != nullptr) st = check(qw);
    if (st != MXFP4_OK) return st;
    Device dev;
    st = device(&dev);
    if (st != MXFP4_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows > 0)
        st = launch(qx, w != nullptr ? &qw : nullptr, dev, s);
    else if (w != nullptr)
        st = launch(qw, nullptr, dev, s);
    return st == MXFP4_OK ? launch(y, dev, s) : st;
}

mxfp4_status mxfp4_grouped_backward(const mxfp4_grouped_linear* l, const void* dy, int64_t lddy, const int32_t* offsets,
                                    int64_t rows, mxfp4_stream_t stream) {
    if (l == nullptr || offsets == nullptr) return MXFP4_ERR_INVALID_ARG;
    const int64_t E = l->groups, N = l->N, K = l->K;
    const Quantize q{dy, rows, N, lddy, nullptr, offsets, E, rows,
                     {l->dy_blobs[0], l->dy_blobs[1], l->dy_blobs[2], l->dy_blobs[3]}};
    if (rows > 0 && (!q.blob[2] || !l->w_blobs[2] || !l->x_blobs[2])) return MXFP4_ERR_INVALID_ARG;
    const mxfp4_out_dtype out = static_cast<mxfp4_out_dtype>(l->out_dtype);
    const Product dx{MXFP4_GROUPED_DGRAD, q.blob[0], q.blob[1], l->w_blobs[2], l->w_blobs[3], offsets, E, rows, N, K,
                     l->dx, K, out};
    const Product dw{MXFP4_GROUPED_WGRAD, q.blob[2], q.blob[3], l->x_blobs[2], l->x_blobs[3], offsets, E, rows, N, K,
                     l->dw, K, out};
    mxfp4_status st = check(dx);
    if (st == MXFP4_OK) st = check(dw);
    if (st == MXFP4_OK) st = check(q);
    if (st != MXFP4_OK) return st;
    Device dev;
    st = device(&dev);
    if (st != MXFP4_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows > 0) st = launch(q, nullptr, dev, s);
    if (st == MXFP4_OK) st = launch(dx, dev, s);
    return st == MXFP4_OK ? launch(dw, dev, s) : st;
}

}  // extern "C"
