// launch_experts.h -- internal interface of the few tokens' layer of experts between its C entry and its
// kernel.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mxfp4.h"

namespace mxfp4 {

// Head of the workspace: where the grid meets, zero between calls.
struct ExpertsSync {
    uint32_t arrived[3];
    uint32_t left;
};

// What a product multiplies.
struct ExpertsSide {
    CUtensorMap map;           // the codes as [rows of all experts, bytes of a row], boxes of 64 bytes of 16 rows, 64-byte swizzle, zero fill
    const uint8_t* codes;
    const uint8_t* scales;
    int32_t rows, k;           // of an expert's weights
    int32_t tiles, slices;     // units of an expert, slices of a unit
    int32_t step, apart;       // a unit's rows: 16 from step * its tile on, below `half`, and 16 from `apart` further on
    int32_t half;
    int32_t pitch, groups;     // of a row of its activations in shared memory: bytes from one to the next, 16-byte pieces
    uint32_t by_tiles, by_slices, by_groups;   // what divides by them
    int32_t down;              // the second product
};

struct ExpertsArgs {
    ExpertsSide side[2];       // W1's, W2's
    const uint16_t* x;         // bf16 [tokens, dim], row pitch ldx
    int64_t ldx;
    const void* logits;        // [tokens, experts], row pitch ldl
    int64_t ldl;
    uint16_t* y;               // bf16 [tokens, dim], row pitch ldy
    int64_t ldy;
    ExpertsSync* sync;
    float* weights;            // [tokens * top_k]: of the choices,
    uint16_t* ids;             // and which experts they are
    uint16_t* lowered;         // fp16 [tokens, dim rounded up to 128]: x times a power of two for each row,
    float* backs;              // [tokens]: which undoes it
    float* h;                  // [tokens * top_k, inner]: the activations between the two products,
    uint32_t* tops;            // [tokens * top_k]: their largest finite magnitudes, as bits; zero between calls
    float* part;               // [tokens * top_k, dim]: the second product's rows, weighted
    uint32_t* err;
    int32_t tokens;
    int32_t experts;
    int32_t top_k;
    int32_t dim;
    int32_t inner;
    int32_t logits_f32;
    int32_t normalize;
    int32_t passes_rows;       // routed rows that one pass over the weights takes: 8 or 16
    int32_t stages;            // slices on their way to shared memory, for each warp: 2 to 4
};

}  // namespace mxfp4
