// pdl.cuh -- programmatic dependent launch: a kernel that may start while the one
// before it in the stream still runs.
#pragma once

#include <cuda_runtime.h>

namespace tcq {

// Lets the next kernel of the stream start once every CTA of this one has got here
// (or ended); it sees none of this kernel's results before its own pdl_wait.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Waits until the kernel before this one in the stream has ended and its results are
// visible (at once when this kernel was launched in the plain way).  A kernel that
// starts early waits before it ends, so that ends keep the stream's order.
// What the kernel before wrote is read past L1 (__ldcg, TMA): __ldg is for data that does
// not change while a kernel runs, and this one was running.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches `kernel`; with `early` it may start before the kernel ahead of it ends.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool early, A... args)
{
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace tcq
