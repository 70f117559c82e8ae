// launch_adamw.h -- internal interface of the AdamW step between its host side (adamw.cu's C
// entry) and its kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxfp4.h"

namespace mxfp4 {

constexpr int kAdamwBlock = 128;     // elements that share the scale of an 8-bit moment
constexpr int kAdamwUnit = 1024;     // elements of a CTA's unit of work
constexpr int kAdamwFew = 40;        // tensors of the small launch's table,
constexpr int kAdamwMany = 320;      // and of the large one's (a kernel parameter: 22 of 32 KB)

template <int kCap>
struct AdamwArgs {
    mxfp4_adamw_tensor t[kCap];
    int32_t end[kCap];               // units of the tensors up to and with this one
    int32_t count;
    float beta1, one_beta1, beta2, one_beta2, eps, weight_decay;
    float lr, c1, c2, grad_scale;    // c = 1 - beta^step
    const float* dynamic;            // or null: lr, c1, c2, grad_scale (stochastic: and the step) in device memory
    int32_t first;                   // stochastic: tensors with elements before t[0] in the call,
    uint32_t step;                   // the step's number
    uint64_t seed;                   // and the key
    const float* grad_factor;        // or null: multiplies the gradients' scale
};

}  // namespace mxfp4
