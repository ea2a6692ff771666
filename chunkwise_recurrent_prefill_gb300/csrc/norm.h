// Group norm with an activation, channels last: the problem as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

struct NormProblem {
    const void *x, *gate, *dy;          // gate may be null; dy in the backward pass only
    const float *w, *b;                 // [C] or null
    void *y, *dx, *dgate;               // [N, L, C] contiguous
    float *mean, *rstd;                 // [N, G]: written forward (or null), read backward
    float *dw, *db;                     // [C] or null
    int64_t N, L, C, G;
    int64_t x_n, x_l, gate_n, gate_l, dy_n, dy_l;   // element strides
    float eps;
    int act, io;
};

size_t norm_workspace_bytes(const NormProblem &p, bool backward, int num_sms);
cudaError_t launch_norm_fwd(const NormProblem &p, void *ws, int num_sms, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormProblem &p, void *ws, int num_sms, cudaStream_t s);

}  // namespace gla
