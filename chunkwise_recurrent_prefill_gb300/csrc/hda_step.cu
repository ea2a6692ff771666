// One token of linear attention with one decay per head, on pages of a pool of states:
//     S <- e^decay S + k^T v,    o = scale q S        (per row and head)
// The state is read and written once: HBM bandwidth bounds a batch, latency a single row.
#include <cuda_bf16.h>

#include "gla_internal.h"
#include "hda_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 16;  // state rows a thread loads before it stores them

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// CTA = (row, head, kCols value columns). A thread owns four columns of every kRows-th key row and
// moves them with 16-byte accesses; the sums over the key rows are added in shared memory in a
// fixed order. Columns of 128 keep whole rows of 512 bytes together; a call of few rows and heads
// takes 32, so that four times as many SMs share it (16 states of 128 x 128: 5.2 us against 6.7).
// Measured: 240 rows of 16 heads of 128 x 128 (512 MB of states and vectors) 79 us in the kernel, 84
// per call, 6.0 TB/s or 89 % of a plain copy's rate.
template <typename T, int kCols>
__global__ void __launch_bounds__(kThreads, 2)
hda_step_kernel(const __grid_constant__ HdaStep p, unsigned int *err) {
    constexpr int kQuads = kCols / 4, kRows = kThreads / kQuads;
    constexpr int kLoad = kCols == 128 ? kBatch : 4;
    __shared__ float4 part[kRows][kQuads];
    extern __shared__ float rows[];   // [2][Dk]: k and q
    const int row0 = threadIdx.x / kQuads, quad = threadIdx.x % kQuads;
    const int r = blockIdx.x / (unsigned)p.H, h = blockIdx.x % (unsigned)p.H;
    const int col = blockIdx.y * kCols + 4 * quad;
    const bool in = col < p.Dv;
    T *op = static_cast<T *>(p.o) + ((int64_t)r * p.H + h) * p.Dv + col;
    const int64_t slot = p.slots ? p.slots[r] : r;
    if (slot < 0 || slot >= p.P) {   // an empty row (uniform over the CTA)
        if (slot >= p.P && threadIdx.x == 0) atomicOr(err, kDevErrPages);
        if (row0 == 0 && in)
            for (int j = 0; j < 4; ++j) put(op + j, 0.f);
        return;
    }
    auto head = [&](const HdaTensor &t) {
        return static_cast<const T *>(t.p) + r * t.b + (h / ((int)p.H / t.heads)) * t.h;
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
    for (int d0 = row0; d0 < p.Dk; d0 += kRows * kLoad) {
        float4 sv[kLoad];
#pragma unroll
        for (int j = 0; j < kLoad; ++j) {
            const int d = d0 + j * kRows;
            sv[j] = (d < p.Dk && in) ? *reinterpret_cast<const float4 *>(Sp + (int64_t)d * p.Dv)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < kLoad; ++j) {
            const int d = d0 + j * kRows;
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
    part[row0][quad] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (row0 == 0 && in) {
        float4 sum = part[0][quad];
#pragma unroll 8
        for (int w = 1; w < kRows; ++w) {
            sum.x += part[w][quad].x;
            sum.y += part[w][quad].y;
            sum.z += part[w][quad].z;
            sum.w += part[w][quad].w;
        }
        put(op, p.scale * sum.x);
        put(op + 1, p.scale * sum.y);
        put(op + 2, p.scale * sum.z);
        put(op + 3, p.scale * sum.w);
    }
}

}  // namespace

template <typename T>
static void run_step(const HdaStep &p, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    const size_t smem = 2 * (size_t)p.Dk * sizeof(float);
    const int64_t ctas = p.R * p.H * ((p.Dv + 127) / 128);
    if (ctas >= num_sms)
        hda_step_kernel<T, 128><<<dim3((unsigned)(p.R * p.H), (unsigned)((p.Dv + 127) / 128)), kThreads, smem, s>>>(
            p, dev_err);
    else
        hda_step_kernel<T, 32><<<dim3((unsigned)(p.R * p.H), (unsigned)((p.Dv + 31) / 32)), kThreads, smem, s>>>(
            p, dev_err);
}

cudaError_t launch_hda_step(const HdaStep &p, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    if (p.io == 0) run_step<__nv_bfloat16>(p, num_sms, dev_err, s);
    else run_step<float>(p, num_sms, dev_err, s);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
