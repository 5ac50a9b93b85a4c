// Kernels of one call that follow one another: the next one's blocks are placed
// while the last ones of the one before run, and wait there until all of it is
// done and its writes are seen.  What this saves is the launch (about 1.5 us a
// kernel).  Only between kernels of one call: the first is an ordinary launch.
#pragma once
#include <cuda_runtime.h>

namespace tq {

// In a kernel launched with launch_next: before anything else.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// In the one before: once all its blocks are here, the next one's may be placed.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, const A &...args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace tq
