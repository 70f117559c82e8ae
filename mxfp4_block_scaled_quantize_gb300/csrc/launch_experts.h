// launch_experts.h -- internal interface of the few tokens' layer of experts between its C entry and its
// kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxfp4.h"

namespace mxfp4 {

struct ExpertsArgs {
    const uint16_t* x;         // bf16 [tokens, dim], row pitch ldx
    int64_t ldx;
    const void* logits;        // [tokens, experts], row pitch ldl
    int64_t ldl;
    const uint8_t* q;          // codes of this kernel's weights,
    const uint8_t* s;          // and their scales
    float* h;                  // [tokens * top_k, inner]: the activations between the two products
    float* part;               // [tokens * top_k, dim]: the second product's rows, weighted
    uint32_t* done;            // a counter for each 32 columns of y, zero between calls
    uint16_t* y;               // bf16 [tokens, dim], row pitch ldy
    int64_t ldy;
    int32_t tokens;
    int32_t experts;
    int32_t top_k;
    int32_t dim;
    int32_t inner;
    int32_t logits_f32;
    int32_t normalize;
    // of this kernel's product
    int32_t rows;              // rows of an expert's weights,
    int32_t k;                 // their length,
    int32_t tiles;             // units in an expert's rows,
    int32_t passes_rows;       // routed rows that one pass over the weights takes
    int32_t stages;            // slices on their way to shared memory, for each warp: 2 or 4
};

}  // namespace mxfp4
