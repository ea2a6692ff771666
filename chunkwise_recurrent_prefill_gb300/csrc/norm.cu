// Group norm with an activation, channels last (forward and backward).
#include <cuda_bf16.h>

#include "gla_internal.h"
#include "norm.h"

namespace gla {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float act_of(float u, int act) {
    if (act == 1) return u / (1.f + expf(-u));
    if (act == 2) return 0.5f * u * (1.f + erff(u * 0.70710678f));
    return u;
}
__device__ __forceinline__ float act_grad(float u, int act) {
    if (act == 1) {
        const float s = 1.f / (1.f + expf(-u));
        return s * (1.f + u * (1.f - s));
    }
    if (act == 2)
        return 0.5f * (1.f + erff(u * 0.70710678f)) + u * expf(-0.5f * u * u) * 0.39894228f;
    return 1.f;
}

// Sum over the block, the same on every thread (a fixed order).
__device__ __forceinline__ float block_sum(float v, float *sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) s += sh[i];
    return s;
}

// One CTA per (entry, group): mean, then the squared deviations from it, then the output.
template <typename T>
__global__ void norm_fwd_kernel(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kThreads / 32];
    const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, cg = p.C / p.G, m = p.L * cg;
    const T *x = static_cast<const T *>(p.x) + n * p.x_n + g * cg;
    float s = 0.f;
    for (int64_t e = threadIdx.x; e < m; e += kThreads) s += get(x + e / cg * p.x_l + e % cg);
    const float mean = block_sum(s, sh) / (float)m;
    s = 0.f;
    for (int64_t e = threadIdx.x; e < m; e += kThreads) {
        const float d = get(x + e / cg * p.x_l + e % cg) - mean;
        s = fmaf(d, d, s);
    }
    const float rstd = 1.f / sqrtf(block_sum(s, sh) / (float)m + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[blockIdx.x] = mean;
        if (p.rstd) p.rstd[blockIdx.x] = rstd;
    }
    for (int64_t e = threadIdx.x; e < m; e += kThreads) {
        const int64_t l = e / cg, c = g * cg + e % cg;
        float u = (get(x + l * p.x_l + e % cg) - mean) * rstd;
        u = fmaf(u, p.w ? p.w[c] : 1.f, p.b ? p.b[c] : 0.f);
        float y;
        if (p.gate) y = u * act_of(get(static_cast<const T *>(p.gate) + n * p.gate_n + l * p.gate_l + c), p.act);
        else y = act_of(u, p.act);
        put(static_cast<T *>(p.y) + (n * p.L + l) * p.C + c, y);
    }
}

struct Grad {
    float xh, du, dz;
};
template <typename T>
__device__ __forceinline__ Grad grad_at(const NormProblem &p, int64_t n, int64_t l, int64_t c,
                                        float mean, float rstd) {
    Grad r;
    r.xh = (get(static_cast<const T *>(p.x) + n * p.x_n + l * p.x_l + c) - mean) * rstd;
    const float u = fmaf(r.xh, p.w ? p.w[c] : 1.f, p.b ? p.b[c] : 0.f);
    const float dy = get(static_cast<const T *>(p.dy) + n * p.dy_n + l * p.dy_l + c);
    if (p.gate) {
        const float z = get(static_cast<const T *>(p.gate) + n * p.gate_n + l * p.gate_l + c);
        r.du = dy * act_of(z, p.act);
        r.dz = dy * u * act_grad(z, p.act);
    } else {
        r.du = dy * act_grad(u, p.act);
        r.dz = 0.f;
    }
    return r;
}

template <typename T>
__global__ void norm_bwd_kernel(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kThreads / 32];
    const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, cg = p.C / p.G, m = p.L * cg;
    const float mean = p.mean[blockIdx.x], rstd = p.rstd[blockIdx.x];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t e = threadIdx.x; e < m; e += kThreads) {
        const int64_t c = g * cg + e % cg;
        const Grad r = grad_at<T>(p, n, e / cg, c, mean, rstd);
        const float d = r.du * (p.w ? p.w[c] : 1.f);
        s1 += d;
        s2 = fmaf(d, r.xh, s2);
    }
    s1 = block_sum(s1, sh) / (float)m;
    s2 = block_sum(s2, sh) / (float)m;
    for (int64_t e = threadIdx.x; e < m; e += kThreads) {
        const int64_t l = e / cg, c = g * cg + e % cg, at = (n * p.L + l) * p.C + c;
        const Grad r = grad_at<T>(p, n, l, c, mean, rstd);
        const float d = r.du * (p.w ? p.w[c] : 1.f);
        put(static_cast<T *>(p.dx) + at, rstd * (d - s1 - r.xh * s2));
        if (p.gate) put(static_cast<T *>(p.dgate) + at, r.dz);
    }
}

// One CTA per channel: dw and db.
template <typename T>
__global__ void norm_dw_kernel(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kThreads / 32];
    const int64_t c = blockIdx.x, g = c / (p.C / p.G);
    float sw = 0.f, sb = 0.f;
    for (int64_t e = threadIdx.x; e < p.N * p.L; e += kThreads) {
        const int64_t n = e / p.L;
        const Grad r = grad_at<T>(p, n, e % p.L, c, p.mean[n * p.G + g], p.rstd[n * p.G + g]);
        sw = fmaf(r.du, r.xh, sw);
        sb += r.du;
    }
    sw = block_sum(sw, sh);
    sb = block_sum(sb, sh);
    if (threadIdx.x == 0) {
        if (p.dw) p.dw[c] = sw;
        if (p.db) p.db[c] = sb;
    }
}

template <typename T>
cudaError_t run_fwd(const NormProblem &p, cudaStream_t s) {
    norm_fwd_kernel<T><<<(unsigned)(p.N * p.G), kThreads, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t run_bwd(const NormProblem &p, cudaStream_t s) {
    norm_bwd_kernel<T><<<(unsigned)(p.N * p.G), kThreads, 0, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (!p.dw && !p.db) return e;
    norm_dw_kernel<T><<<(unsigned)p.C, kThreads, 0, s>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

size_t norm_workspace_bytes(const NormProblem &, bool, int) { return 0; }

cudaError_t launch_norm_fwd(const NormProblem &p, void *, int, cudaStream_t s) {
    return p.io == 0 ? run_fwd<__nv_bfloat16>(p, s) : run_fwd<float>(p, s);
}

cudaError_t launch_norm_bwd(const NormProblem &p, void *, int, cudaStream_t s) {
    return p.io == 0 ? run_bwd<__nv_bfloat16>(p, s) : run_bwd<float>(p, s);
}

}  // namespace gla
