// launch_grad_norm.h -- internal interface of the gradients' norm between its C entry and its kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "mxfp4.h"

namespace mxfp4 {

constexpr int kGradUnitBytes = 16384;  // a CTA's unit of work
constexpr int kGradThreads = 256;
constexpr int kGradCtasPerSm = 4;
constexpr int kGradMaxSms = 256;
constexpr int kGradSlots = kGradCtasPerSm * kGradMaxSms;   // partial sums of one launch
constexpr int kGradFew = 48;           // tensors of the small launch's table,
constexpr int kGradMany = 1280;        // and of the large one's (a kernel parameter: 25 of 32 KB)

constexpr int kGradLaunches = MXFP4_GRAD_MAX_TENSORS / kGradMany + 1;

// Head of the workspace; the launches' partial sums follow it.
struct GradHead {
    uint32_t done;                     // CTAs that have left their sum: zero between calls
    uint32_t pad[63];
};

template <int kCap>
struct GradArgs {
    mxfp4_grad_tensor t[kCap];
    int32_t end[kCap];                 // units of the tensors up to and with this one
    int32_t count;
    GradHead* head;
    double* partial;                   // of the whole call; this launch's start at `slot`
    int32_t slot;
    int32_t slots;                     // of the whole call: the CTA that fills the last one adds them up
    double max_norm;
    float* out;                        // norm, factor
};

}  // namespace mxfp4
