// grad_norm_launches.cu -- the host part of the gradients' norm, with its launches noted instead of made.
#include <cuda_runtime.h>

#include "launch.h"
#include "launch_grad_norm.h"

// One launch: its CTAs, and of its table the tensors, their elements and units, and where its partial sums go.
struct Noted {
    int64_t ctas, tensors, elements, units, slot, slots;
};

namespace {

Noted noted[256];
int64_t count = 0;

template <int kCap>
void note(int64_t ctas, const mxfp4::GradArgs<kCap>& a) {
    Noted n = {ctas, a.count, 0, a.count > 0 ? a.end[a.count - 1] : 0, a.slot, a.slots};
    for (int i = 0; i < a.count; ++i) n.elements += a.t[i].n;
    noted[count++] = n;
}
void note(int64_t ctas, float*) { noted[count++] = {ctas, 0, 0, 0, 0, 0}; }

template <typename Kernel, typename Args>
cudaError_t launch_noted(const cudaLaunchConfig_t* cfg, Kernel, const Args& a) {
    if (cfg->gridDim.x == 0) return cudaErrorInvalidConfiguration;
    note(cfg->gridDim.x, a);
    return cudaSuccess;
}

}  // namespace

#define cudaLaunchKernelEx launch_noted
#include "grad_norm.cu"

namespace mxfp4 {
int device_info(int* sms, uint32_t** err) {
    *sms = 152;
    *err = nullptr;
    return MXFP4_OK;
}
}  // namespace mxfp4

// The launches of a call of mxfp4_grad_norm with these tensors, into `out`; their number in `launches`.
extern "C" int launches_of(int32_t tensors, const mxfp4_grad_tensor* t, int32_t flags, Noted* out, int64_t* launches) {
    size_t bytes = 0;
    mxfp4_grad_norm_workspace_bytes(tensors, &bytes);
    count = 0;
    const mxfp4_status st = mxfp4_grad_norm(tensors, t, flags, 1.0, reinterpret_cast<float*>(0x1000), reinterpret_cast<void*>(0x1000), bytes, nullptr);
    for (int64_t i = 0; i < count; ++i) out[i] = noted[i];
    *launches = count;
    return st;
}
