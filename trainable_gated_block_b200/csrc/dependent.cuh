// Launches that overlap the latency of a launch with the end of the kernel
// in front of it in the stream (programmatic dependent launch). Every kernel
// launched this way calls after_previous() before it touches memory, which
// waits until that kernel has finished and its writes are visible: only the
// placement of the CTAs comes early. It reads global memory by ordinary loads, which
// that wait orders: not by the read-only path (__ldg, ld.global.nc, or const
// __restrict__ parameters, which the compiler reads so), which is for memory that
// nobody writes while the kernel runs, and the kernel in front may write what this one
// reads when it has been placed already. In a stream of calls this saves one to two
// microseconds a kernel (a ragged append 20.5 -> 18.5 us). Early CTAs go
// where the kernel in front leaves room first: a persistent grid of several CTAs an
// SM needs shared memory that lets no more of them onto an SM (norm + rotation of 8k
// tokens: 30.5 us, without 32.5). kEarly = false is for grids that lose all the same
// (the append of an 8k prompt behind a kernel of many small CTAs: 41.1, early 55.4).
#pragma once

#include <cuda_runtime.h>

namespace sas {

__device__ __forceinline__ void after_previous() {
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <bool kEarly = true, int kCluster = 1, typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (kEarly) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (kCluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = kCluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace sas
