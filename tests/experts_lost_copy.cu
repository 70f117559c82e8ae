// experts_lost_copy.cu -- the kernel of the few tokens' experts with one stage's barrier that expects an arrival more than there is:
// the wait for it runs out, after 20 ms.  Counts the tensor copies that each warp asks for.
#include <cuda_runtime.h>

#include "launch.h"
#include "launch_experts.h"
#include "ptx.cuh"

namespace mxfp4 {
namespace {
__device__ int lost_cta = -1, lost_thread = -1;   // whose barrier: the thread that sets it up
__device__ int copies[256 * 16];

__device__ __forceinline__ void set_up(uint32_t bar, uint32_t count) {
    const bool more = static_cast<int>(blockIdx.x) == lost_cta && static_cast<int>(threadIdx.x) == lost_thread;
    mbar_init(bar, more ? count + 1 : count);
}
__device__ __forceinline__ void count_and_load(uint32_t to, const CUtensorMap* map, int x, int y, uint32_t bar) {
    atomicAdd(&copies[blockIdx.x * 16 + (threadIdx.x >> 5)], 1);
    tma_load_2d(to, map, x, y, bar);
}
}  // namespace
}  // namespace mxfp4

#define mbar_init set_up
#define tma_load_2d count_and_load
#define mbar_wait(bar, parity, err, site, abort) mbar_wait(bar, parity, err, site, abort, 20000000ull)
#include "experts.cu"

// From here on the barrier that thread `thread` of CTA `cta` sets up is never complete (-1: none is so), and the copies are counted anew.
extern "C" int lose(int cta, int thread) {
    static const int zeros[256 * 16] = {};
    if (cudaMemcpyToSymbol(mxfp4::lost_cta, &cta, sizeof(cta)) != cudaSuccess) return 1;
    if (cudaMemcpyToSymbol(mxfp4::lost_thread, &thread, sizeof(thread)) != cudaSuccess) return 1;
    return cudaMemcpyToSymbol(mxfp4::copies, zeros, sizeof(zeros)) != cudaSuccess;
}

extern "C" int counted(int* out) { return cudaMemcpyFromSymbol(out, mxfp4::copies, 256 * 16 * sizeof(int)) != cudaSuccess; }
