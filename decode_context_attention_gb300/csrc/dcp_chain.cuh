// dcp_chain.cuh -- kernels of one call whose launch and start overlap the one before.
#pragma once

#include <cuda_runtime.h>

namespace dcp {

// Programmatic stream serialisation: chain_wait() returns when the kernel before is done and
// its writes are visible, chain_release() lets the next one start (its CTAs as SMs have room).
// At least one CTA of every kernel of the chain waits, so that the last one's end is the end
// of all; a kernel that releases before it waits would let the next one see what the one
// before it has not finished.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... P, class... A>
cudaError_t launch_chained(void (*kernel)(P...), unsigned ctas, int threads, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace dcp
