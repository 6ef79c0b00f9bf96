// Shared memory limits of kernels, and one launch, with clusters where asked, that may begin while the
// kernel before it in the stream ends (the kernels wait for it themselves, pdl_wait_previous).
#pragma once

#include "common.cuh"

namespace nvfp4 {

// Lets `kernel` take `bytes` of dynamic shared memory on the current device.  The limit is
// the kernel's, not the call's: it only ever rises, so that calls of other sizes, from other
// threads, do not take it away between this and the launch.
nvfp4_status allow_smem(const void* kernel, size_t bytes, const char* what);

inline nvfp4_status launch_kernel(const void* kernel, dim3 grid, dim3 block, size_t smem, unsigned cluster, void** args,
                                  cudaStream_t stream, const char* fn) {
    if (smem > 8 * 1024)                                    // with what the kernel declares, past 48 KB
        if (nvfp4_status st = allow_smem(kernel, smem, fn)) return st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return check_cuda(cudaLaunchKernelExC(&cfg, kernel, args), fn);
}

}  // namespace nvfp4
