// Linear attention with one decay per head: the problem as the kernels see it.
//
// The forward and the three gradients are one map. With l = e^decay, over the tokens in order
// (or in reverse order),
//     out_t = a_out x_t S_t,     S_t = l S_{t-1} + a_in y_t^T z_t
// reversed: S_t = S'_{t+1} + a_in y_t^T z_t, out_t = a_out x_t S_t, S'_t = l S_t (the state a
// reversed pass starts from and returns already carries the decay of the step it stands at).
//     forward : x = q,   y = k,   z = v    S = h0     (a_in, a_out) = (1, scale)
//     dq      : x = d_o, y = v,   z = k    S = h0^T   (1, scale)
//     dk      : x = v,   y = d_o, z = q    S = dhT^T  reversed, (scale, 1)
//     dv      : x = k,   y = q,   z = d_o  S = dhT    reversed, (scale, 1); returns dh0
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gla {

struct HdaTensor {
    const void *p;
    int64_t b, t, h;        // element strides
    int heads;              // state head s of H reads head s / (H / heads)
};

struct HdaLin {
    HdaTensor x, y, z;      // x, y: Dx wide; z: Dz wide
    const float *init;      // [B,H,Dx,Dz], or [B,H,Dz,Dx] with init_t; null: zero
    float *fin;             // the same for the state at the end (fin_t); null: not wanted
    int init_t, fin_t;
    void *out;              // [B,T,H,Dz] contiguous: the caller's type, or float (out_f32)
    int out_f32;
    int Dx, Dz;
    float a_in, a_out;
    int rev;
};

struct HdaProblem {
    const float *decay;     // [H] log-decays
    int64_t B, T, H;
    int io;                 // GLA_IO_BF16 / GLA_IO_F32
    int n;                  // maps: 1 (forward) or 3 (gradients, in the order dq, dk, dv)
    HdaLin lin[3];
};

// Sum over the state heads that share a head: in [BT, H, D] float -> out [BT, heads, D].
struct HdaShare {
    const float *in;
    void *out;
    int heads, D;
};

// l^n = e^(n g): the product is formed in two parts, so that the result is good to a few 2^-24
// of itself (the rounding of n g alone would cost 2^-24 |n g|). 1 for n = 0, whatever g is.
__device__ __forceinline__ float decay_pow(float g, float n) {
    if (n == 0.f) return 1.f;
    const float p = n * g;
    if (!(p > -100.f)) return expf(p);      // below (or NaN): the correction has no meaning
    return expf(p) * (1.f + fmaf(n, g, -p));
}

// splits: segments of a sequence, 0 = by the rule beside exact_plan.
size_t hda_exact_workspace_bytes(const HdaProblem &p, int splits, int num_sms);
cudaError_t launch_hda_exact(const HdaProblem &p, int splits, int num_sms, void *ws, cudaStream_t s);
cudaError_t launch_hda_share(const HdaShare *parts, int n, int64_t BT, int64_t H, int io,
                             cudaStream_t s);
struct HdaStep {
    HdaTensor q, k, v;
    const float *decay;
    float scale;
    float *S;
    const int *slots;       // null: row r is page r
    void *o;
    int64_t R, P, H;
    int Dk, Dv, io;
};
cudaError_t launch_hda_step(const HdaStep &p, int num_sms, unsigned int *dev_err, cudaStream_t s);

// Tensor-core path (bf16, Dx and Dz of every map in {64, 128}).
bool hda_tc_supported(const HdaProblem &p);
size_t hda_tc_workspace_bytes(const HdaProblem &p, int splits, int num_sms);
cudaError_t launch_hda_tc(const HdaProblem &p, int splits, int num_sms, void *ws,
                          unsigned int *dev_err, cudaStream_t s);

}  // namespace gla
