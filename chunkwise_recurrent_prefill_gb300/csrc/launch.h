// Kernel launches of the operators around a recurrent layer (host code).
#pragma once

#include <cuda_runtime.h>

#include "gla_internal.h"

namespace gla {

// Launches and counts. dependent: the kernel is scheduled while the one before it in the stream still runs, and
// waits for it itself (pdl_wait_prerequisites).
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool dependent, cudaStream_t s,
                   const A &...args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
