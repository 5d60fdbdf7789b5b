// Launches of the kernels around the cache: programmatic dependents of the kernel before them,
// with a cluster where asked, and the limit of their dynamic shared memory.
#pragma once
#include <cuda_runtime.h>

#include "once.h"

namespace lora {

template <typename... P, typename... A>
cudaError_t start(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                  const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const P &>(args)...);
}

template <typename K>
cudaError_t allow_shared(OncePerDevice &once, K kernel, size_t bytes)
{
    return once([=] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)); });
}

}  // namespace lora
