// Depthwise causal convolution with an activation: the problem as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

struct ConvProblem {
    const void *x, *dy;
    int64_t x_b, x_t, dy_b, dy_t;       // element strides
    const float *w, *bias;              // [C, W], [C] or null
    const void *s0, *dsT;               // [B, W - 1, C] or null
    void *y, *sT;                       // [B, T, C], [B, W - 1, C] or null
    void *dx, *ds0;                     // the same
    float *dw, *dbias;                  // [C, W], [C] or null
    int64_t B, T, C;
    int W, act, io;
    // one token
    void *S;                            // [P, W - 1, C]
    const int *slots;
    int64_t P;
};

cudaError_t launch_conv_fwd(const ConvProblem &p, int num_sms, cudaStream_t s);
size_t conv_bwd_workspace_bytes(const ConvProblem &p, int num_sms);
cudaError_t launch_conv_bwd(const ConvProblem &p, void *ws, int num_sms, cudaStream_t s);
cudaError_t launch_conv_step(const ConvProblem &p, unsigned int *dev_err, cudaStream_t s);

}  // namespace gla
