// art_stream.cuh -- how the cache operators' kernels follow one another on a
// stream: every one is launched as a programmatic dependent of the kernel
// before it, so that its CTAs can take their places while that one ends.
//
// Each thread of such a kernel calls follow() before it touches global memory
// and, whatever it has to do, before it ends: follow() returns when the kernel
// before has ended and its writes are visible, and a kernel that ended
// earlier would let its own successor start too early.  lead(), after it, lets
// the successor's CTAs come while this kernel still runs: the attention's
// first kernel does that for the one that joins its parts (1 us).  Elsewhere it
// cost time, waiting CTAs take places that the last ones of the kernel before
// still need (an append of 2.5k tokens 7.4 us with it and 5.3 without, an
// eviction 39.3 and 35.6).  Only reads of inputs that no kernel of the same
// call writes may stand before follow(), in a kernel whose predecessor is of
// the same call and leads after its own follow(); they go past the L1 cache.
// Read-only loads (__ldg) have no place here: the kernel before may still be
// writing when this one's life begins.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace art_stream {

__device__ __forceinline__ void follow() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void lead() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// SMs of the current device (a B200's where it cannot be asked)
inline int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Launches fn(a) in clusters of `cluster` CTAs, after what the stream holds.
template <typename A>
cudaError_t launch(void (*fn)(A), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &a, int cluster = 1)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, fn, a);
}

}  // namespace art_stream
