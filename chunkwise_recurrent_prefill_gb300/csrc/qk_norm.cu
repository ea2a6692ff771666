// Norm of queries and keys for each head with the position rotation in the same pass:
//     n = x r w,   r = (s sum x^2 + eps)^-1/2;   pairs (a, b) of n -> (a cos - b sin, b cos + a sin)
// and its gradient, with g the gradient of n (the rotation's transpose of the output's) times w and
// xh = x r:
//     dx = r (g - xh s sum(g xh)),   dw = sum over tokens and heads of (g / w) xh
// Every value is read once and written once, so HBM bandwidth bounds it.
#include <algorithm>

#include "elem.cuh"
#include "gla_internal.h"
#include "qk_norm.h"

namespace gla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float sum_warp(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// r from the sum of squares. Where that leaves the range in which its digits are good, sum2(scale), the
// sum of squares of the values times a power of two, takes its place (the same in all lanes).
template <typename F>
__device__ __forceinline__ float norm_factor(float ss, float s, float eps, const F &sum2) {
    const float v = fmaf(s, ss, eps);
    if (v >= 1e-30f && v <= 1e37f) return rsqrtf(v);
    const float f = v < 1.f ? 0x1p100f : 0x1p-100f;
    return f * rsqrtf(fmaf(s, sum2(f), eps * f * f));
}

// One head of a token, as the warps go through them: token-major, queries before keys.
struct Row {
    int64_t token, b, t;
    int which, head;
};
__device__ __forceinline__ Row row_of(const QkProblem &p, int64_t id) {
    const int heads = p.t[0].heads + p.t[1].heads;
    Row r;
    r.token = id / heads;
    const int h = (int)(id - r.token * heads);
    r.which = h >= p.t[0].heads;
    r.head = h - (r.which ? p.t[0].heads : 0);
    r.b = r.token / p.T;
    r.t = r.token - r.b * p.T;
    return r;
}

// The row of the tables of a token, or -1 if its position is outside of them.
__device__ __forceinline__ int64_t position(const QkProblem &p, const Row &r, unsigned int *err) {
    const int64_t at = p.positions ? p.positions[r.token] : r.t;
    if (p.R == 0 || (at >= 0 && at < p.P)) return at;
    if (threadIdx.x % 32 == 0) atomicOr(err, kDevErrPages);
    return -1;
}

// A warp per head, a lane every 32nd pair, whatever the sizes and alignment.
template <typename T>
__global__ void __launch_bounds__(kThreads)
qk_plain_fwd(const __grid_constant__ QkProblem p, unsigned int *err) {
    const int lane = threadIdx.x % 32;
    const int64_t id = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
    const Row r = row_of(p, id);
    if (r.b >= p.B) return;
    const QkHeads &h = p.t[r.which];
    const T *x = static_cast<const T *>(h.x) + r.b * h.x_b + r.t * h.x_t + r.head * h.x_h;
    const int64_t at = r.token * h.heads + r.head;
    T *out = static_cast<T *>(h.out) + at * p.D;
    const int64_t pos = position(p, r, err);
    if (p.R > 0 && pos < 0) {
        for (int i = lane; i < p.D; i += 32) put(out + i, 0.f);
        if (h.r && lane == 0) h.r[at] = 0.f;
        return;
    }
    float f = 1.f;
    if (p.norm) {
        auto sum2 = [&](float scale) {
            float ss = 0.f;
            for (int i = lane; i < p.D; i += 32) {
                const float v = get(x + i) * scale;
                ss = fmaf(v, v, ss);
            }
            return sum_warp(ss);
        };
        f = norm_factor(sum2(1.f), p.norm == 1 ? 1.f / (float)p.D : 1.f, p.eps, sum2);
        if (h.r && lane == 0) h.r[at] = f;
    }
    auto value = [&](int i) { return get(x + i) * f * (h.w ? h.w[i] : 1.f); };
    const int half = p.R / 2;
    for (int i = lane; i < half; i += 32) {
        const int ia = p.pairs ? 2 * i : i, ib = p.pairs ? 2 * i + 1 : i + half;
        const float a = value(ia), b = value(ib), c = p.cos[pos * half + i], s = p.sin[pos * half + i];
        put(out + ia, fmaf(a, c, -(b * s)));
        put(out + ib, fmaf(b, c, a * s));
    }
    for (int i = p.R + lane; i < p.D; i += 32) put(out + i, value(i));
}

// Sums of a CTA's rows go to part[blockIdx.x][2][D].
template <typename T>
__global__ void __launch_bounds__(kThreads)
qk_plain_bwd(const __grid_constant__ QkProblem p, float *part, unsigned int *err) {
    extern __shared__ float sums[];         // [2][kWarps][D]
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (int i = threadIdx.x; i < 2 * kWarps * p.D; i += kThreads) sums[i] = 0.f;
    __syncthreads();
    const int64_t rows = p.B * p.T * (p.t[0].heads + p.t[1].heads);
    for (int64_t id = (int64_t)blockIdx.x * kWarps + warp; id < rows; id += (int64_t)gridDim.x * kWarps) {
        const Row r = row_of(p, id);
        const QkHeads &h = p.t[r.which];
        const T *x = static_cast<const T *>(h.x) + r.b * h.x_b + r.t * h.x_t + r.head * h.x_h;
        const T *go = static_cast<const T *>(h.go) + r.b * h.g_b + r.t * h.g_t + r.head * h.g_h;
        const int64_t at = r.token * h.heads + r.head;
        T *out = static_cast<T *>(h.out) + at * p.D;
        const int64_t pos = position(p, r, err);
        if (p.R > 0 && pos < 0) {
            for (int i = lane; i < p.D; i += 32) put(out + i, 0.f);
            continue;
        }
        const float f = p.norm ? h.r[at] : 1.f, s = p.norm == 1 ? 1.f / (float)p.D : 1.f;
        const int half = p.R / 2;
        // g / w of both values of pair i
        auto back = [&](int i, float &ga, float &gb, int &ia, int &ib) {
            ia = p.pairs ? 2 * i : i;
            ib = p.pairs ? 2 * i + 1 : i + half;
            const float a = get(go + ia), b = get(go + ib), c = p.cos[pos * half + i], sn = p.sin[pos * half + i];
            ga = fmaf(a, c, b * sn);
            gb = fmaf(b, c, -(a * sn));
        };
        auto weight = [&](int i) { return h.w ? h.w[i] : 1.f; };
        float dot = 0.f;
        if (p.norm) {
            float *dw = sums + (r.which * kWarps + warp) * p.D;
            auto one = [&](int i, float g) {
                const float gx = g * (get(x + i) * f);
                dw[i] += gx;
                dot = fmaf(gx, weight(i), dot);
            };
            for (int i = lane; i < half; i += 32) {
                float ga, gb;
                int ia, ib;
                back(i, ga, gb, ia, ib);
                one(ia, ga);
                one(ib, gb);
            }
            for (int i = p.R + lane; i < p.D; i += 32) one(i, get(go + i));
            dot = sum_warp(dot) * s;
        }
        auto write = [&](int i, float g) {
            put(out + i, p.norm ? f * (g * weight(i) - get(x + i) * f * dot) : g);
        };
        for (int i = lane; i < half; i += 32) {
            float ga, gb;
            int ia, ib;
            back(i, ga, gb, ia, ib);
            write(ia, ga);
            write(ib, gb);
        }
        for (int i = p.R + lane; i < p.D; i += 32) write(i, get(go + i));
    }
    if (!part) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        const int which = i / p.D, d = i - which * p.D;
        float s = 0.f;
        for (int k = 0; k < kWarps; ++k) s += sums[(which * kWarps + k) * p.D + d];
        part[(int64_t)blockIdx.x * 2 * p.D + i] = s;
    }
}

// dwq and dwk from the CTAs' parts, added in their order.
__global__ void __launch_bounds__(kThreads)
qk_sums_kernel(const __grid_constant__ QkProblem p, const float *part, int parts) {
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= 2 * p.D) return;
    float s = 0.f;
    for (int k = 0; k < parts; ++k) s += part[(int64_t)k * 2 * p.D + i];
    float *dw = p.t[i / p.D].dw;
    if (dw) dw[i % p.D] = s;
}

int64_t rows_of(const QkProblem &p) { return p.B * p.T * (p.t[0].heads + p.t[1].heads); }

int bwd_parts(const QkProblem &p, int num_sms) {
    return (int)std::min<int64_t>((rows_of(p) + kWarps - 1) / kWarps, 4 * num_sms);
}

}  // namespace

cudaError_t launch_qk_fwd(const QkProblem &p, int, unsigned int *dev_err, cudaStream_t s) {
    const unsigned grid = (unsigned)((rows_of(p) + kWarps - 1) / kWarps);
    if (p.io == 0) qk_plain_fwd<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, dev_err);
    else qk_plain_fwd<float><<<grid, kThreads, 0, s>>>(p, dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

size_t qk_bwd_workspace_bytes(const QkProblem &p, int num_sms) {
    return p.norm ? (size_t)bwd_parts(p, num_sms) * 2 * p.D * sizeof(float) : 0;
}

template <typename T>
static cudaError_t run_bwd(const QkProblem &p, float *part, int parts, unsigned int *err, cudaStream_t s) {
    const size_t smem = 2 * kWarps * (size_t)p.D * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(qk_plain_bwd<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    qk_plain_bwd<T><<<parts, kThreads, smem, s>>>(p, part, err);
    return cudaGetLastError();
}

cudaError_t launch_qk_bwd(const QkProblem &p, void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    const int parts = bwd_parts(p, num_sms);
    float *part = p.norm && (p.t[0].dw || p.t[1].dw) ? static_cast<float *>(ws) : nullptr;
    cudaError_t e = p.io == 0 ? run_bwd<__nv_bfloat16>(p, part, parts, dev_err, s)
                              : run_bwd<float>(p, part, parts, dev_err, s);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (part) {
        qk_sums_kernel<<<(2 * p.D + kThreads - 1) / kThreads, kThreads, 0, s>>>(p, part, parts);
        e = cudaGetLastError();
        if (e == cudaSuccess) count_launches(1);
    }
    return e;
}

}  // namespace gla
