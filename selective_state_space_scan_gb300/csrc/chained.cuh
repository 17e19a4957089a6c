// Kernels of one call that follow one another on its stream: the next one's blocks may come up, and do what does not
// touch memory that the one before writes, while the one before still ends.  A chained kernel calls wait_for_earlier()
// in every thread before it reads or writes such memory; a call's first kernel is launched as any other, after all that
// was on the stream.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace selscan {

__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may come up as soon as every block has called this or ended.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(std::forward<A>(args))...);
}

}  // namespace selscan
