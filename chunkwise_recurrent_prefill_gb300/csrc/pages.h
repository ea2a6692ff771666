// Pages of a pool of states: the plan and copy kernels' launchers.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

struct PagePool {
    void *pool;
    int64_t P, page_bytes;
    int *table;
    int64_t R, M;
    int *free_stack, *count;
};

// ws: so many bytes, 16-byte aligned (the moves planned on the device, and marks).
size_t pages_fork_workspace(const PagePool &p, int64_t n);
size_t pages_free_workspace(const PagePool &p);
size_t pages_compact_workspace(const PagePool &p);
cudaError_t launch_pages_copy(const PagePool &p, const int *src, const int *dst, int64_t n,
                              int num_sms, unsigned int *dev_err, cudaStream_t s);
cudaError_t launch_pages_fork(const PagePool &p, const int *parents, const int *children, int64_t n,
                              void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s);
cudaError_t launch_pages_free(const PagePool &p, const int *rows, int64_t n, void *ws,
                              unsigned int *dev_err, cudaStream_t s);
cudaError_t launch_pages_compact(const PagePool &p, void *ws, int num_sms, unsigned int *dev_err,
                                 cudaStream_t s);

}  // namespace gla
