// pa_launch.cuh -- kernel launch as a programmatic dependent of the previous
// kernel on the stream: its launch overlaps that kernel's tail, and the
// kernel waits for it (griddepcontrol.wait) before touching memory.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace pa {

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_smem(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                            Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, Args&&... args) {
    return launch_pdl_smem(kernel, grid, block, 0, stream, std::forward<Args>(args)...);
}

}  // namespace pa
