// Selective state space scan: the problem as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

struct SsmRows {
    const void *p;
    int64_t b, t;           // element strides
};

struct SsmProblem {
    SsmRows u, dt, z, Bm, Cm, go;       // z.p may be null; go (d_o) in the backward pass only
    const float *A;                     // [C, N]
    const float *D, *dt_bias;           // [C] or null
    const float *h0, *dhT;              // [B, C, N] or null
    void *o;                            // [B, T, C] contiguous
    float *hT;                          // [B, C, N] or null
    void *du, *ddt, *dz, *dBm, *dCm;    // backward, contiguous; dz may be null
    float *dA, *dD, *dbias, *dh0;       // dD, dbias, dh0 may be null
    int64_t B, T, C, G;
    int N, softplus, io;
    // one token
    float *S;                           // [P, C, N]
    const int *slots;
    int64_t P;
};

size_t ssm_fwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms);
size_t ssm_bwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms);
cudaError_t launch_ssm_fwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err,
                           cudaStream_t s);
cudaError_t launch_ssm_bwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err,
                           cudaStream_t s);
cudaError_t launch_ssm_step(const SsmProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s);

}  // namespace gla
