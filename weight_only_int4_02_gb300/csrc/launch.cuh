// Launch of the serving step's kernels, chained like the GEMMs by programmatic dependent launch.
#pragma once
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace w4a16 {

// The first statement of each such kernel. Its CTAs may be put on the SMs while the kernel before it on the
// stream drains (1.5 to 2 us less between two small kernels); they touch no global memory until that
// kernel has finished, and only then let the next kernel in, so that a GEMM behind this one, which reads its
// weights ahead of its own wait, still finds whatever was written before this kernel.
__device__ __forceinline__ void chained_kernel()
{
    wait_prior_grid();
    launch_dependents();
}

template <typename P>
cudaError_t launch_chained(void (*kernel)(P), unsigned grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t stream,
                           const P& p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace w4a16
