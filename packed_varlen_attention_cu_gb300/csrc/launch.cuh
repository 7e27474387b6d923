// launch.cuh -- dependent launches: kernels that may be launched while the kernel before them in
// the stream still runs.
#pragma once

#include <cuda_runtime.h>

namespace pva {

// Dependent launches.  A kernel of the cache and beam calls may be launched while the kernel before
// it in the stream runs out, and waits for its end: a chain of short kernels (append,
// attention, join) pays less for its launches (0.3 to 1 us each; letting the next kernel
// start any earlier than the last blocks' exit was no better and cost the long ones 1%).
// All reads and writes come after the wait, and no thread block leaves without having
// waited, so that the end of a kernel is the end of all before it.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                                const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// The kernel of the backward that makes D lets the next one start early: once every block has come here (or
// has ended), blocks of the kernel launched after this one take the multiprocessors that are free, and wait.
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace pva
