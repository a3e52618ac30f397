// mxfp4_launch.h -- launching the MXFP4 kernels.
#pragma once

#include <cuda_runtime.h>

namespace fgemm {
namespace mx {

// Every MXFP4 kernel is a programmatic dependent of the kernel before it in its stream: its
// CTAs may come to the SMs while that one runs, set up their barriers and tensor memory, and
// wait (griddepcontrol.wait) until it has completed before they access what it may write or
// read.  Only then do they let the next kernel do the same, so no kernel ends before the one
// before it has, and the next one's wait covers them all.  All threads wait before their first
// access to global memory, but for one warp: the product behind fgemm_mxfp4_linear's quantising
// asks for the weight first, which that kernel, itself past its wait, does not write.
// Back to back in a graph, 256^3 products take 2.5 us in place of 3.4, seven tokens through
// 1237 -> 1001 (two kernels) 5.3 in place of 7.3.
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
