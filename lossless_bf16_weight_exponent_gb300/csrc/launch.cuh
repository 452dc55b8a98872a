// launch.cuh - programmatic dependent launch: a kernel starts while the one before it on the stream drains, sets itself
// up, and waits before it touches anything that one may write or read.  Every CTA waits, also one without work, so that
// a grid that has ended vouches for all grids before it.
// What an earlier kernel may write is read by plain loads alone: it changes during such a kernel's life, while __ldg (the
// non-coherent path) is for memory that does not.  Only the frozen compressed weights go that way.
#pragma once

#include <cuda_runtime.h>

#include "per_device.h"

namespace uw {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// allows a kernel this much dynamic shared memory on the current device (an attribute of each device's own)
template <typename... P>
cudaError_t allow_shared(OncePerDevice &once, void (*kernel)(P...), size_t bytes)
{
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    return (cudaError_t)once(device, [&] { return (int)cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
}

// cluster > 0: CTAs per cluster along x
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st,
                             const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute la[2];
    la[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    la[0].val.programmaticStreamSerializationAllowed = 1;
    la[1].id = cudaLaunchAttributeClusterDimension;
    la[1].val.clusterDim.x = cluster;
    la[1].val.clusterDim.y = la[1].val.clusterDim.z = 1;
    cfg.attrs = la;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace uw
