// Launching a kernel whose workspace head has to start at zero, without paying for the
// clearing: a one-block kernel clears it, and the kernel proper is launched as its programmatic
// dependent, so that it starts while the other still runs.  The clearing kernel itself starts when
// everything before it in the stream is done, so the dependent may read its inputs at once; only
// before it touches the cleared words does it wait (head_cleared()), and once at its end, so that
// it is not done before they are cleared.  A 256-byte memset before
// each launch cost about 3 us of a 12 us call.
#pragma once

#include "common.cuh"
#include "host_common.h"

namespace dspark {

__device__ __forceinline__ void head_cleared() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

namespace {
__global__ void clear_head(uint4* head, int n) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < n; i += blockDim.x) head[i] = make_uint4(0, 0, 0, 0);
}
}  // namespace

// set_status for kernels launched so.
static __device__ __noinline__ void tell(StatusBlock* st, uint32_t code, uint32_t detail) {
    head_cleared();
    set_status(st, code, detail);
}

// Clears `bytes` (a multiple of 16) at `head`, then launches `kernel`; nothing else may come between.
template <class... P, class... A>
dspark_status_t launch_cleared(void* head, size_t bytes, void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                               cudaStream_t s, A&&... args) {
    clear_head<<<1, 256, 0, s>>>(static_cast<uint4*>(head), static_cast<int>(bytes / 16));
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
        cudaGetLastError();
        return DSPARK_ERR_CUDA;
    }
    return launch_status();
}

}  // namespace dspark
