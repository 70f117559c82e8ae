// launch_norm.h -- internal interface of layer norm between its C entry and its kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxfp4.h"

namespace mxfp4 {

constexpr int kNormWarpRowDim = 512;     // rows of up to this many elements are one warp's in either pass
// Rows that a CTA has on their way to shared memory, at most.
constexpr int kNormStagesForward = 3;
constexpr int kNormStagesBackward = 4;
constexpr int kNormStages = 4;

// CTAs that share the rows of a backward pass, each of which leaves a partial row of dw and db: as many as 152 SMs hold at a time.
inline int norm_chunks(int64_t dim) { return dim <= kNormWarpRowDim ? 608 : 152; }
inline int64_t norm_slots(int64_t dim) { return 2 * norm_chunks(dim); }
constexpr int64_t kNormLeastRows = 4;    // of a CTA, where there are few: a partial row costs as much as two rows of x

// How rows are read and written: norm_row.cuh.
enum NormAccess { kNormSingle, kNormWide, kNormShifted };

struct NormArgs {
    const void* x;
    const void* dy;          // backward
    const void* weight;      // [samples, dim] or null
    const void* bias;
    void* y;                 // backward: dx
    float* mean;
    float* rstd;
    float* partial_w;        // backward: [chunks of all samples, dim], or null
    float* partial_b;
    int64_t ldx, lddy, ldy;
    int64_t rows;
    int64_t sample_rows;     // rows of a sample
    int64_t chunk_rows;      // backward: rows of a CTA, all of one sample, every period-th from its first on
    int32_t chunks;          // backward: CTAs of a sample, of which the first `period` start at its first rows
    int32_t period;          // rows from one to the next that is shifted alike: 1 but for kNormShifted
    NormAccess access;
    int32_t dim;
    float eps;
    int32_t w_f32;
    int32_t w_wide;          // weight and bias start at multiples of 16 bytes
    int32_t add_one;
    int32_t stages;          // rows on their way to shared memory (its ring), where rows are copied there
    uint32_t* err;
};

struct NormReduceArgs {
    const float* partial[2]; // [samples * chunks, dim]
    float* out[2];           // [samples, dim]
    int32_t count;           // of the two
    int32_t chunks;
    int32_t dim;
    int64_t samples;
};

cudaError_t launch_norm_forward(const NormArgs& a, bool f32, int sms, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormArgs& a, bool f32, int64_t ctas, cudaStream_t stream);
cudaError_t launch_norm_reduce(const NormReduceArgs& a, cudaStream_t stream);

}  // namespace mxfp4
