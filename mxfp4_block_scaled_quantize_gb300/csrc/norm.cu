// norm.cu -- layer norm's C entries: checks, and how a backward pass shares its rows out.
#include <cmath>
#include <cstring>

#include "launch.h"
#include "launch_norm.h"

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 40;

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool shape_ok(int64_t rows, int64_t dim, int64_t samples) {
    return rows >= 0 && rows <= kMaxRows && dim >= 1 && dim <= MXFP4_NORM_MAX_DIM && samples >= 1 && samples <= kMaxRows &&
           rows % samples == 0;
}

// One row alone may have any pitch.
bool pitch_ok(int64_t ld, int64_t dim, int64_t rows) { return rows <= 1 || (ld >= dim && ld <= (int64_t{1} << 40)); }

// Would a written row of `out` be another row's input in `in`?  A row is read whole before it is written, so `out` may be `in` itself; and
// the two may lie side by side in rows of one pitch.
bool mixed(const void* in, int64_t ldi, const void* out, int64_t ldo, int64_t rows, int64_t dim, int64_t size) {
    if (rows == 0 || (in == out && (rows == 1 || ldi == ldo))) return false;
    const __int128 a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out), row = dim * size;
    const __int128 steps = rows - 1;
    if (a + steps * ldi * size + row <= b || b + steps * ldo * size + row <= a) return false;
    if (rows == 1 || ldi != ldo) return true;
    const __int128 pitch = static_cast<__int128>(ldi) * size, between = ((b - a) % pitch + pitch) % pitch;
    return between < row || pitch - between < row;
}

// How the kernels may access these tensors of rows (null: not there), and the rows from one to the next that is shifted alike.
// Shifted accesses cost every row some masks and a launch its edge rows; they are for bf16 rows that CTAs take, and, of a
// backward pass, for many elements.  us shifted and single: forward 8192 rows of 4100 39 and 71, 16000 of 6001 87 and 161, 1111 of
// 1001 4.9 and 6.1; backward 1111 of 1001 10.2 and 9.0, 4000 of 777 13.9 and 14.9, 2000 of 2001 15.2 and 15.8, 8192 of 1001 20.3 and
// 22.8, 100 of 5001 13.4 and 12.0, 600 of 7001 24.1 and 20.3, 8192 of 4100 68 and 84, 16000 of 6001 131 and 175; fp32, 3000 of 2050,
// 13.3 and 14.0 forward, 26.5 and 23 backward; rows of 250, a warp's, 13.1 and 7.7.
void set_access(mxfp4::NormArgs* a, bool f32, const void* const* rows, const int64_t* pitches, int count) {
    const int64_t size = f32 ? 4 : 2;
    uintptr_t base = 0;
    bool wide = a->dim % 8 == 0, alike = true;
    a->w_wide = aligned_to(a->weight, 16) && aligned_to(a->bias, 16);
    int64_t step = 0;   // bytes from a row to the next, modulo 16; of one row alone: none
    for (int i = 0; i < count; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(rows[i]) & 15u;
        const int64_t by = a->rows > 1 ? (pitches[i] % 16) * size % 16 : 0;
        if (i == 0) {
            base = at;
            step = by;
        }
        alike = alike && at == base && by == step;
        wide = wide && at == 0 && by == 0;
    }
    a->period = 1;
    if (wide) {
        a->access = mxfp4::kNormWide;
    } else if (alike && !f32 && a->dim > mxfp4::kNormWarpRowDim && a->dim + 7 <= MXFP4_NORM_MAX_DIM &&
               (count == 2 || a->rows >= (int64_t{1} << (a->dim <= 4096 ? 21 : 23)) / a->dim)) {
        a->access = mxfp4::kNormShifted;
        while (step * a->period % 16 != 0) a->period *= 2;
    } else {
        a->access = mxfp4::kNormSingle;
    }
}

}  // namespace

extern "C" {

mxfp4_status mxfp4_layer_norm_workspace_bytes(int64_t dim, size_t* bytes) {
    if (dim < 1 || dim > MXFP4_NORM_MAX_DIM || bytes == nullptr) return MXFP4_ERR_INVALID_ARG;
    *bytes = 2 * static_cast<size_t>(mxfp4::norm_slots(dim)) * static_cast<size_t>(dim) * sizeof(float);
    return MXFP4_OK;
}

mxfp4_status mxfp4_layer_norm(const void* x, int64_t rows, int64_t dim, int64_t ldx, const void* weight, const void* bias,
                              int64_t samples, double eps, int32_t flags, void* y, int64_t ldy, float* mean, float* rstd,
                              mxfp4_stream_t stream) {
    if (!shape_ok(rows, dim, samples) || !pitch_ok(ldx, dim, rows) || !pitch_ok(ldy, dim, rows) || (flags & ~7) ||
        !(eps >= 0.0) || !std::isfinite(static_cast<float>(eps)) || (rows > 0 && (x == nullptr || y == nullptr)) ||
        (mean == nullptr) != (rstd == nullptr))
        return MXFP4_ERR_INVALID_ARG;
    const uintptr_t xe = flags & MXFP4_NORM_X_F32 ? 4 : 2, we = flags & MXFP4_NORM_W_F32 ? 4 : 2;
    if (!aligned_to(x, xe) || !aligned_to(y, xe) || !aligned_to(weight, we) || !aligned_to(bias, we) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4))
        return MXFP4_ERR_MISALIGNED;
    if (mixed(x, ldx, y, ldy, rows, dim, xe)) return MXFP4_ERR_INVALID_ARG;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK || rows == 0) return static_cast<mxfp4_status>(st);
    mxfp4::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldy = ldy;
    a.rows = rows;
    a.sample_rows = rows / samples;
    a.dim = static_cast<int32_t>(dim);
    a.eps = static_cast<float>(eps);
    a.w_f32 = flags & MXFP4_NORM_W_F32 ? 1 : 0;
    a.add_one = flags & MXFP4_NORM_ADD_ONE ? 1 : 0;
    a.err = err;
    const void* const tensors[2] = {x, y};
    const int64_t pitches[2] = {ldx, ldy};
    set_access(&a, flags & MXFP4_NORM_X_F32, tensors, pitches, 2);
    return mxfp4::launch_norm_forward(a, flags & MXFP4_NORM_X_F32, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MXFP4_OK
               : MXFP4_ERR_CUDA;
}

mxfp4_status mxfp4_layer_norm_backward(const void* dy, int64_t lddy, const void* x, int64_t rows, int64_t dim, int64_t ldx,
                                       const void* weight, int64_t samples, int32_t flags, const float* mean, const float* rstd,
                                       void* dx, int64_t lddx, float* dw, float* db, void* workspace, size_t workspace_bytes,
                                       mxfp4_stream_t stream) {
    if (!shape_ok(rows, dim, samples) || !pitch_ok(ldx, dim, rows) || !pitch_ok(lddy, dim, rows) || !pitch_ok(lddx, dim, rows) ||
        (flags & ~7) || (rows > 0 && (!dy || !x || !mean || !rstd || !dx)))
        return MXFP4_ERR_INVALID_ARG;
    const uintptr_t xe = flags & MXFP4_NORM_X_F32 ? 4 : 2, we = flags & MXFP4_NORM_W_F32 ? 4 : 2;
    if (!aligned_to(x, xe) || !aligned_to(dy, xe) || !aligned_to(dx, xe) || !aligned_to(weight, we) || !aligned_to(mean, 4) ||
        !aligned_to(rstd, 4) || !aligned_to(dw, 4) || !aligned_to(db, 4) || !aligned_to(workspace, 16))
        return MXFP4_ERR_MISALIGNED;
    if (mixed(x, ldx, dx, lddx, rows, dim, xe) || mixed(dy, lddy, dx, lddx, rows, dim, xe)) return MXFP4_ERR_INVALID_ARG;
    mxfp4::NormArgs a;
    std::memset(&a, 0, sizeof(a));
    a.rows = rows;
    a.dim = static_cast<int32_t>(dim);
    a.weight = weight;
    const void* const tensors[3] = {x, dy, dx};
    const int64_t pitches[3] = {ldx, lddy, lddx};
    set_access(&a, flags & MXFP4_NORM_X_F32, tensors, pitches, 3);
    // Each CTA its rows of one sample, shifted alike; norm_chunks(dim) CTAs at most, if the samples are not more.
    const int64_t sample_rows = rows / samples;
    int64_t chunk_rows = 1, chunks = 1;
    auto split = [&] {
        const int64_t alike = cdiv(sample_rows, a.period), most = mxfp4::norm_chunks(dim) / (samples * a.period);
        const int64_t even = most > 1 ? cdiv(alike, most) : alike;
        chunk_rows = even > mxfp4::kNormLeastRows ? even : mxfp4::kNormLeastRows;
        chunks = rows > 0 ? a.period * cdiv(alike, chunk_rows) : 1;
    };
    split();
    if (a.period > 1 && samples * chunks > mxfp4::norm_slots(dim)) {   // many short samples: their partial rows would not fit
        a.access = mxfp4::kNormSingle;
        a.period = 1;
        split();
    }
    const int64_t ctas = samples * chunks;
    const bool partial = chunks > 1 && (dw != nullptr || db != nullptr);
    size_t need = 0;
    if (partial && (mxfp4_layer_norm_workspace_bytes(dim, &need) != MXFP4_OK || workspace == nullptr || workspace_bytes < need))
        return MXFP4_ERR_INVALID_ARG;
    if (ctas > 0x7FFFFFFF) return MXFP4_ERR_INVALID_ARG;
    int sms = 0;
    uint32_t* err = nullptr;
    const int st = mxfp4::device_info(&sms, &err);
    if (st != MXFP4_OK) return static_cast<mxfp4_status>(st);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        const size_t bytes = static_cast<size_t>(samples) * static_cast<size_t>(dim) * sizeof(float);
        for (float* const v : {dw, db})
            if (v != nullptr && cudaMemsetAsync(v, 0, bytes, s) != cudaSuccess) return MXFP4_ERR_CUDA;
        return MXFP4_OK;
    }
    a.x = x;
    a.dy = dy;
    a.y = dx;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    float* const w = static_cast<float*>(workspace);
    a.partial_w = dw == nullptr ? nullptr : partial ? w : dw;
    a.partial_b = db == nullptr ? nullptr : partial ? w + mxfp4::norm_slots(dim) * dim : db;
    a.ldx = ldx;
    a.lddy = lddy;
    a.ldy = lddx;
    a.sample_rows = sample_rows;
    a.chunk_rows = chunk_rows;
    a.chunks = static_cast<int32_t>(chunks);
    a.w_f32 = flags & MXFP4_NORM_W_F32 ? 1 : 0;
    a.add_one = flags & MXFP4_NORM_ADD_ONE ? 1 : 0;
    a.err = err;
    if (mxfp4::launch_norm_backward(a, flags & MXFP4_NORM_X_F32, ctas, s) != cudaSuccess) return MXFP4_ERR_CUDA;
    if (!partial) return MXFP4_OK;
    mxfp4::NormReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    for (int i = 0; i < 2; ++i) {
        float* const out = i == 0 ? dw : db;
        if (out == nullptr) continue;
        r.partial[r.count] = i == 0 ? a.partial_w : a.partial_b;
        r.out[r.count++] = out;
    }
    r.chunks = a.chunks;
    r.dim = a.dim;
    r.samples = samples;
    return mxfp4::launch_norm_reduce(r, s) == cudaSuccess ? MXFP4_OK : MXFP4_ERR_CUDA;
}

}  // extern "C"
