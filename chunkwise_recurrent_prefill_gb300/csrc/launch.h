// Kernel launches of the operators around a recurrent layer (host code).
#pragma once

#include <cuda_runtime.h>

#include "gla_internal.h"

namespace gla {

// Launches and counts. The kernel may be scheduled while the one before it in the stream still runs, whoever's that
// is: its first access to global memory comes after pdl_wait_prerequisites(), which all of its CTAs call, so that a kernel
// that is done implies that those before it are. (Between calls that follow each other this hides the launch:
// 16384 x 4096 channels of a convolution 52.7 -> 50.2 us a call.)
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const A &...args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
