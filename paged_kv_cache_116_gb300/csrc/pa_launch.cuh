// pa_launch.cuh -- kernel launch as a programmatic dependent of the previous
// kernel on the stream: its launch overlaps that kernel's tail, and the
// kernel waits for it (griddepcontrol.wait) before touching memory.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace pa {

// Raises a kernel's limit of dynamic shared memory to the most that any of its
// launches asks for.  The limit belongs to the kernel, not to the launch: set
// to one call's own size, a smaller call of another host thread would lower it
// before this one's launch, which is then refused.
inline cudaError_t allow_smem(const void* kernel, size_t most) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

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
