// chain.cuh -- launches of kernels that may be scheduled while the kernel before them in the stream
// still runs (programmatic stream serialization).  Such a kernel calls chain_wait() before its first
// access to global memory, in every thread: it returns when the kernel before has ended and its
// writes are there, so stream order holds as usual and only the latency of the launch is hidden.
// chain_release() lets the next such kernel be scheduled once all blocks of this one have started.
#pragma once
#include <cuda_runtime.h>

namespace dr {
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
}  // namespace dr
