// Kernel launches of the operators around a recurrent layer (host code).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

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

// Lets a kernel have all of a CTA's shared memory, once for each device. (Not what a call needs: another thread's call of
// the kernel could set a lower limit before the launch.)
template <auto kKernel>
cudaError_t allow_shared() {
    static std::atomic<uint64_t> done{0};
    int dev = 0, most = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    cudaFuncAttributes attr{};
    e = cudaFuncGetAttributes(&attr, kKernel);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)attr.sharedSizeBytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace gla
