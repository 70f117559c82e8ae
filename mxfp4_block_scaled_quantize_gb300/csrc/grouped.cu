// grouped.cu -- host side of the linears grouped by expert (include/mxfp4.h): argument checks,
// tensor maps and launches.  Nothing here reads the group offsets: they stay on the device.
#include <cstring>

#include "launch.h"
#include "mxfp4.h"

namespace {

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 512;
constexpr int64_t kTileConstant = 320; // of the cost of a tile, in columns
// Tokens a group, on average, up to which the few-token products run (8 groups, 4096 x 4096: 26.6 us
// against 30.7 at 96 tokens, 34.8 against 30.8 at 192).  The average is all that the host knows; one
// large group among 63 of one token, 2048 x 2048, loses little by it: 45.6 us for 5953 rows by these
// products, 43.4 for 6145 by the others.
constexpr int64_t kFewTokens = 96;

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
    const int64_t tiles = wgrad ? t.groups * cdiv(t.N, 256) * cdiv(t.K, 128)
                                : most_tiles(t.rows, t.groups, t.offsets == nullptr, 128) * cdiv(cols, 256);
    if (tiles > (int64_t{1} << 31) - 1) return MXFP4_ERR_INVALID_ARG;
    return MXFP4_OK;
}

// The elements [rows, packed / 2] of a blob, boxes of box_rows rows x 128 bytes.
bool element_map(CUtensorMap* m, const void* q, int64_t rows, int64_t packed, uint32_t box_rows) {
    return mxfp4::encode_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, static_cast<uint64_t>(packed / 2),
                                static_cast<uint64_t>(rows), static_cast<uint64_t>(packed / 2), 128, box_rows,
                                CU_TENSOR_MAP_SWIZZLE_128B);
}

// Its scales as rows of 128-row atom groups in 8-byte units, boxes of box_groups x 2 atoms.
bool scale_map(CUtensorMap* m, const void* s, int64_t rows, int64_t packed, uint32_t box_groups) {
    return mxfp4::encode_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, s, static_cast<uint64_t>(packed / 128) * 64,
                                static_cast<uint64_t>(rows / 128), static_cast<uint64_t>(packed / 128) * 512, 128,
                                box_groups, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The operand whose rows are the MMA's M, and the one whose rows are its N.
bool m_maps(mxfp4::GroupedGemmArgs* g, const void* q, const void* s, int64_t rows, int64_t packed, int64_t scale_rows) {
    return element_map(&g->amap, q, rows, packed, 128) && scale_map(&g->sfamap, s, scale_rows, packed, 1);
}

bool n_maps(mxfp4::GroupedGemmArgs* g, const void* q, const void* s, int64_t rows, int64_t packed, int64_t scale_rows,
            bool few) {
    for (int i = 0; i < 4; ++i)
        if (!element_map(&g->bmap[i], q, rows, packed, 16u << i)) return false;
    return scale_map(&g->sfbmap, s, scale_rows, packed, few ? 1 : 3);
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

// What a product's kernel may rely on before the launch ahead of it is done: nothing, or that what
// came before that launch is complete, offsets with it, or W's blob too.
enum Ready { kNothing, kOffsets, kOffsetsAndW };

// Columns of the tiles of `strips` strips of `cols` columns each (forward, dgrad: a group's tokens on
// average, all that the host knows of them): the width whose modelled time is least.  The
// tiles go round the clusters in waves, and a tile costs its columns and a constant.  A whole training
// step, as graph replays, at 384, 256 and 128 columns throughout, in us: 64 groups of 384 tokens, 1408 x 2048, 349, 357,
// 425; 8 of 2048, 8192 x 2048, 485, 533, 736; 5 of 222 in fp32 with few tiles to go round 56.0, 53.7,
// 53.9, where the rule's own mixture takes 53.1.  The constant came from the first two: at 256 the
// rule took 256 columns for the second one's dgrad, and that step 502 us; it now takes 481.
int32_t tile_width(int64_t strips, int64_t cols, int64_t clusters) {
    int32_t best = 384;
    int64_t least = INT64_MAX;
    for (int32_t width = 384; width >= 128; width -= 128) {
        const int64_t tiles = cdiv(cols, width);
        const int64_t time = cdiv(strips * tiles, clusters) * (cdiv(cols, tiles) + kTileConstant);
        if (time < least) {
            least = time;
            best = width;
        }
    }
    return best;
}

mxfp4_status launch(const Product& t, const Device& dev, cudaStream_t stream, Ready ready = kNothing) {
    const bool wgrad = t.form == MXFP4_GROUPED_WGRAD;
    const bool f32 = t.out == MXFP4_OUT_F32;
    const int64_t esize = f32 ? 4 : 2;
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
    const bool few = !wgrad && t.rows <= t.groups * kFewTokens;
    bool maps;
    if (t.form == MXFP4_GROUPED_FWD) {
        maps = m_maps(&g, t.b_q, t.b_s, t.groups * t.N, kp, t.groups * np) && n_maps(&g, t.a_q, t.a_s, t.rows, kp, cap, few);
        g.atoms = static_cast<int32_t>(kp / 128);
        g.a_step_rows = static_cast<int32_t>(t.N);
        g.a_step_groups = static_cast<int32_t>(np / 128);
        g.m_rows = static_cast<int32_t>(t.N);
    } else if (t.form == MXFP4_GROUPED_DGRAD) {
        maps = m_maps(&g, t.b_q, t.b_s, t.K, t.groups * np, kp) && n_maps(&g, t.a_q, t.a_s, t.rows, np, cap, few);
        g.atoms = static_cast<int32_t>(np / 128);
        g.a_step_atoms = static_cast<int32_t>(np / 128);
        g.m_rows = static_cast<int32_t>(t.K);
    } else {
        maps = m_maps(&g, t.a_q, t.a_s, t.N, cap, np) && n_maps(&g, t.b_q, t.b_s, t.K, cap, kp, false);
        g.m_rows = static_cast<int32_t>(t.N);
        g.n_cols = static_cast<int32_t>(t.K);
    }
    if (!maps) return MXFP4_ERR_CUDA;
    g.tiles_m = static_cast<int32_t>(cdiv(g.m_rows, 256));
    const int64_t cols = wgrad ? t.K : g.m_rows;
    g.c_tma = (t.ldc * esize) % 16 == 0 &&
              mxfp4::encode_map_2d(&g.cmap, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t.c,
                                   static_cast<uint64_t>(cols), static_cast<uint64_t>(wgrad ? t.groups * t.N : t.rows),
                                   static_cast<uint64_t>(t.ldc * esize), static_cast<uint32_t>(64 / esize), 32,
                                   CU_TENSOR_MAP_SWIZZLE_64B);
    g.offsets = t.offsets;
    g.groups = static_cast<int32_t>(t.groups);
    g.rows = static_cast<int32_t>(t.rows);
    g.c = t.c;
    g.ldc = t.ldc;
    g.out_f32 = f32 ? 1 : 0;
    g.early_offsets = ready != kNothing;
    g.early_m = ready == kOffsetsAndW;
    g.err = dev.err;
    const int most = mxfp4::gemm_grouped_max_clusters();
    if (most <= 0) return MXFP4_ERR_CUDA;
    g.width = few ? 128 : tile_width(t.groups * g.tiles_m, wgrad ? t.K : cdiv(t.rows, t.groups), most);
    const int64_t tiles = g.tiles_m * (wgrad ? t.groups * cdiv(t.K, g.width) : most_tiles(t.rows, t.groups, equal, 128));
    const int clusters = static_cast<int>(tiles < most ? tiles : most);
    return mxfp4::launch_gemm_grouped(g, wgrad, few, clusters, stream) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
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
    // the quantizers let a launch start only when all before them is complete
    return st == MXFP4_OK ? launch(y, dev, s, rows == 0 ? kNothing : w == nullptr ? kOffsetsAndW : kOffsets) : st;
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
    if (st == MXFP4_OK) st = launch(dx, dev, s, rows > 0 ? kOffsetsAndW : kNothing);
    return st == MXFP4_OK ? launch(dw, dev, s, rows > 0 ? kOffsets : kNothing) : st;
}

}  // extern "C"
