// mxfp4_launch.h -- launching the MXFP4 kernels.
#pragma once

#include <cuda_runtime.h>

namespace fgemm {
namespace mx {

// Every MXFP4 kernel is a programmatic dependent of the kernel before it in its stream: its
// CTAs may come to the SMs while that one ends, set up their barriers and tensor memory, and
// wait (griddepcontrol.wait, all threads, before the first access to global memory) until it
// has completed.  Only then do they let the next kernel do the same.  Kernel after kernel of
// one stream takes 2 us less each that way (256^3 products back to back: 6.2 against 3.9 us);
// and as no kernel ends before the one before it has, the next one's wait covers them all.
// cluster: CTAs of a cluster, or 1.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, unsigned cluster,
                   const A &...args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return e;
}

}  // namespace mx
}  // namespace fgemm
