// Launches that overlap the end of the kernel before.
#pragma once

#include "common.cuh"

namespace gdr {

// The kernels of one call follow each other without draining the GPU between them:
// each lets the next one start once its own blocks have, and every thread that reads
// what an earlier kernel of the call wrote waits for the one before to be complete
// first (the wait also makes those writes visible to its grid; nothing else does).
// Every kernel launched with `after` waits in every block that has work, at its
// start or at its end, so a kernel is complete only when all before it in the call
// are.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... Params, typename... Args>
cudaError_t launch_kernel(bool after, void (*kernel)(Params...), dim3 grid, int threads, size_t smem,
                          cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a;
    c.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

}  // namespace gdr
