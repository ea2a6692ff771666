// One token of linear attention with one decay per head, on pages of a pool of states:
//     S <- e^decay S + k^T v,    o = scale q S        (per row and head)
// The state is read and written once: HBM bandwidth bounds a batch, latency a single row.
#include <cuda_bf16.h>

#include "gla_internal.h"
#include "hda_internal.h"

namespace gla {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 16;  // state rows a warp loads before it stores them

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// CTA = (row, head, 128 value columns). Warp w updates key rows w, w + 8, ...; lane l owns four
// columns and moves them with 16-byte accesses. The per-column sums of the warps are added in
// shared memory in a fixed order.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 2)
hda_step_kernel(const __grid_constant__ HdaStep p, unsigned int *err) {
    __shared__ float4 part[kWarps][32];
    extern __shared__ float rows[];   // [2][Dk]: k and q
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const int col = blockIdx.y * 128 + 4 * lane;
    const bool in = col < p.Dv;
    T *op = static_cast<T *>(p.o) + (r * p.H + h) * p.Dv + col;
    const int64_t slot = p.slots ? p.slots[r] : r;
    if (slot < 0 || slot >= p.P) {   // an empty row (uniform over the CTA)
        if (slot >= p.P && threadIdx.x == 0) atomicOr(err, kDevErrPages);
        if (warp == 0 && in)
            for (int j = 0; j < 4; ++j) put(op + j, 0.f);
        return;
    }
    auto head = [&](const HdaTensor &t) {
        return static_cast<const T *>(t.p) + r * t.b + (h / (p.H / t.heads)) * t.h;
    };
    const T *kp = head(p.k), *qp = head(p.q), *vp = head(p.v) + col;
    for (int d = threadIdx.x; d < p.Dk; d += blockDim.x) {
        rows[d] = get(kp + d);
        rows[p.Dk + d] = get(qp + d);
    }
    const float lam = expf(p.decay[h]);
    __syncthreads();
    float v[4] = {0.f, 0.f, 0.f, 0.f}, acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (in)
        for (int j = 0; j < 4; ++j) v[j] = get(vp + j);
    float *Sp = p.S + (slot * p.H + h) * p.Dk * (int64_t)p.Dv + col;
    for (int d0 = warp; d0 < p.Dk; d0 += kWarps * kBatch) {
        float4 sv[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int d = d0 + j * kWarps;
            sv[j] = (d < p.Dk && in) ? *reinterpret_cast<const float4 *>(Sp + (int64_t)d * p.Dv)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int d = d0 + j * kWarps;
            if (d < p.Dk && in) {
                const float kd = rows[d], qd = rows[p.Dk + d];
                float4 s4;
                s4.x = fmaf(lam, sv[j].x, kd * v[0]);
                s4.y = fmaf(lam, sv[j].y, kd * v[1]);
                s4.z = fmaf(lam, sv[j].z, kd * v[2]);
                s4.w = fmaf(lam, sv[j].w, kd * v[3]);
                *reinterpret_cast<float4 *>(Sp + (int64_t)d * p.Dv) = s4;
                acc[0] = fmaf(qd, s4.x, acc[0]);
                acc[1] = fmaf(qd, s4.y, acc[1]);
                acc[2] = fmaf(qd, s4.z, acc[2]);
                acc[3] = fmaf(qd, s4.w, acc[3]);
            }
        }
    }
    part[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (warp == 0 && in) {
        float4 sum = part[0][lane];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            sum.x += part[w][lane].x;
            sum.y += part[w][lane].y;
            sum.z += part[w][lane].z;
            sum.w += part[w][lane].w;
        }
        put(op, p.scale * sum.x);
        put(op + 1, p.scale * sum.y);
        put(op + 2, p.scale * sum.z);
        put(op + 3, p.scale * sum.w);
    }
}

}  // namespace

cudaError_t launch_hda_step(const HdaStep &p, unsigned int *dev_err, cudaStream_t s) {
    const dim3 grid((unsigned)(p.R * p.H), (unsigned)((p.Dv + 127) / 128));
    const size_t smem = 2 * (size_t)p.Dk * sizeof(float);
    if (p.io == 0) hda_step_kernel<__nv_bfloat16><<<grid, kWarps * 32, smem, s>>>(p, dev_err);
    else hda_step_kernel<float><<<grid, kWarps * 32, smem, s>>>(p, dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
