// Norm of queries and keys for each head, with their rotation: the problem as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

// One of the two tensors.
struct QkHeads {
    const void *x, *go;             // [B, T, heads, D]; go (gradient of the output) backward only
    int64_t x_b, x_t, x_h, g_b, g_t, g_h;   // element strides
    const float *w;                 // [D] or null
    void *out;                      // forward: the output; backward: dx; contiguous
    float *r;                       // [B, T, heads]: written forward (or null), read backward
    float *dw;                      // [D] or null
    int heads;
};

struct QkProblem {
    QkHeads t[2];                   // q, k
    const float *cos, *sin;         // [P, R / 2]
    const int *positions;           // [B, T] or null
    int64_t B, T, P;
    int D, R, norm, pairs, io;
    float eps;
    int stall;                  // test hook: the first load of each warp is never issued
};

cudaError_t launch_qk_fwd(const QkProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s);
size_t qk_bwd_workspace_bytes(const QkProblem &p, int num_sms);
cudaError_t launch_qk_bwd(const QkProblem &p, void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s);

}  // namespace gla
