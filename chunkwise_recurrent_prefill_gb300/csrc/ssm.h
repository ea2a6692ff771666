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
    // Set by the launchers, whose kernels read by TMA: rows of B and C, and the groups of the other inputs, are this
    // many elements apart (N and C / G, or those brought to 16 bytes by a copy), and whether TMA writes.
    int64_t group;
    int row, tma_out;
    int stall;                          // test hook: warp of each ring whose first load is never issued (-1: none)
    // one token
    float *S;                           // [P, C, N]
    const int *slots;
    int64_t P;
};

// any: whatever the alignment of the inputs' pointers (which inputs are copied first depends on it).
size_t ssm_fwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms, bool any);
size_t ssm_bwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms, bool any);
cudaError_t launch_ssm_fwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err,
                           cudaStream_t s);
cudaError_t launch_ssm_bwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err,
                           cudaStream_t s);
cudaError_t launch_ssm_step(const SsmProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s);

}  // namespace gla
