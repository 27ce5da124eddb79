// chained.cuh -- programmatic dependent launch.  A call of several kernels
// launches all but the first as "chained": the blocks of the next kernel may
// be scheduled while the last blocks of the one before still run, so that a
// launch's latency and a kernel's set-up are hidden.  Every kernel of such a
// call waits for the end of the one before it ahead of its first access to
// memory that any kernel of the call writes, and reads that memory with plain
// loads: the read-only path (__ldg, const __restrict__) is for what nobody
// writes while the kernel is resident, and its loads may move ahead of the wait.
#pragma once

#include <cuda_runtime.h>

namespace tg {

__device__ __forceinline__ void wait_for_previous_kernel() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void allow_next_kernel() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// After the wait, by a thread that issues tensor copies: what the kernels before
// wrote with ordinary stores is visible to them.
__device__ __forceinline__ void fence_proxy_async_global() {
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

template <class... P, class... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, unsigned block, cudaStream_t stream,
                           A... args) {
    cudaLaunchConfig_t lc = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    lc.gridDim = grid;
    lc.blockDim = dim3(block, 1, 1);
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kern, P(args)...);
}

}  // namespace tg
