// Depthwise causal convolution with an activation, channels last:
//     a[t] = bias + sum_j w[j] x[t - (W - 1) + j],   y = act(a)
//     da[t] = dy[t] act'(a[t]);  dx[t] = sum_j w[j] da[t + W - 1 - j];  dw[j] = sum_t da[t] x[t - (W - 1) + j]
// Every element is read once and written once, so HBM bandwidth bounds all of it. A thread owns a
// vector of channels and walks over a run of tokens with the last W inputs (and, backwards, the last W
// da) in registers; only the W - 1 inputs around a run are read twice, from L2. Time runs forward
// in both directions: the gradient of token t is complete W - 1 tokens later.
#include <algorithm>

#include "conv.h"
#include "elem.cuh"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 256;

// How the runs and channel vectors share CTAs: lanes (a power of two) threads side by side on the
// channels, kThreads / lanes runs.
struct ConvPlan {
    int lanes;
    int run;            // tokens of a run
    int64_t runs;       // of one sequence
};

// A thread's vector of the input at time t (of its own sequence): before the first token, s0.
template <typename T, int kV>
struct Inputs {
    const T *x;         // of the sequence and the first channel
    const T *s0;
    int64_t x_t, C;
    int W;
    using R = typename Pack<T, kV>::raw;
    __device__ __forceinline__ R at(int64_t t) const {
        if (t >= 0) return *reinterpret_cast<const R *>(x + t * x_t);
        return s0 ? *reinterpret_cast<const R *>(s0 + (t + W - 1) * C) : R{};
    }
};

template <typename T, int kV, int W>
__device__ __forceinline__ void load_weights(const ConvProblem &p, int64_t c, float (&w)[W][kV], float (&b)[kV]) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = __ldg(p.w + (c + v) * W + j);
        b[v] = p.bias ? __ldg(p.bias + c + v) : 0.f;
    }
}

template <typename T, int kV, int W>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const __grid_constant__ ConvProblem p, const ConvPlan pl) {
    constexpr int kBatch = 8;           // tokens loaded at a time
    using P = Pack<T, kV>;
    using R = typename P::raw;
    const int lane = threadIdx.x % pl.lanes;
    const int64_t c = ((int64_t)blockIdx.y * pl.lanes + lane) * kV;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / pl.lanes) + threadIdx.x / pl.lanes;
    const int64_t b = id / pl.runs;
    if (c >= p.C || b >= p.B) return;
    const int64_t t0 = (id - b * pl.runs) * pl.run, t1 = min(t0 + pl.run, p.T);
    const int64_t tail = b * (W - 1) * p.C + c;
    const Inputs<T, kV> in{static_cast<const T *>(p.x) + b * p.x_b + c,
                           p.s0 ? static_cast<const T *>(p.s0) + tail : nullptr, p.x_t, p.C, W};
    T *yp = static_cast<T *>(p.y) + (b * p.T + t0) * p.C + c;
    T *sT = p.sT ? static_cast<T *>(p.sT) + tail : nullptr;
    float w[W][kV], bias[kV], win[W][kV];       // win[j]: the input j - (W - 1) tokens from the current one
    load_weights<T, kV, W>(p, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const R r = in.at(t0 - (W - 1) + j);
        P::unpack(r, win[j + 1]);
        // the part of sT that lies before the first token
        if (sT && t0 == 0 && j >= p.T) *reinterpret_cast<R *>(sT + (j - p.T) * p.C) = r;
    }
    const int64_t keep = p.T - (W - 1);         // tokens from here on are part of sT
    for (int64_t t = t0; t < t1; t += kBatch) {
        R raw[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) raw[i] = t + i < t1 ? in.at(t + i) : R{};
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (t + i >= t1) break;
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < kV; ++v) win[j][v] = win[j + 1][v];
            P::unpack(raw[i], win[W - 1]);
            float a[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                a[v] = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) a[v] = fmaf(w[j][v], win[j][v], a[v]);
                a[v] = act_of<T>(a[v], p.act);
            }
            *reinterpret_cast<R *>(yp) = P::pack(a);
            yp += p.C;
            if (sT && t + i >= keep) *reinterpret_cast<R *>(sT + (t + i - keep) * p.C) = raw[i];
        }
    }
}

// Sums of a CTA's runs go to part[blockIdx.x][W + 1][C]: dw, then dbias.
template <typename T, int kV, int W>
__global__ void __launch_bounds__(kThreads)
conv_bwd_kernel(const __grid_constant__ ConvProblem p, const ConvPlan pl, float *part) {
    constexpr int kBatch = 4;
    using P = Pack<T, kV>;
    using R = typename P::raw;
    __shared__ float sums[kThreads][kV];
    const int lane = threadIdx.x % pl.lanes, row = threadIdx.x / pl.lanes, rows = kThreads / pl.lanes;
    const int64_t c = ((int64_t)blockIdx.y * pl.lanes + lane) * kV;
    const int64_t id = (int64_t)blockIdx.x * rows + row;
    const int64_t b = id / pl.runs;
    float w[W][kV], bias[kV], dw[W][kV], db[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    if (c < p.C && b < p.B) {
        load_weights<T, kV, W>(p, c, w, bias);
        const int64_t t0 = (id - b * pl.runs) * pl.run, t1 = min(t0 + pl.run, p.T);
        const int64_t tail = b * (W - 1) * p.C + c;
        const Inputs<T, kV> in{static_cast<const T *>(p.x) + b * p.x_b + c,
                               p.s0 ? static_cast<const T *>(p.s0) + tail : nullptr, p.x_t, p.C, W};
        const T *dyp = static_cast<const T *>(p.dy) + b * p.dy_b + c;
        const T *dsT = p.dsT ? static_cast<const T *>(p.dsT) + tail : nullptr;
        T *dx = static_cast<T *>(p.dx) + b * p.T * p.C + c;
        T *ds0 = p.ds0 ? static_cast<T *>(p.ds0) + tail : nullptr;
        const int64_t keep = p.T - (W - 1);
        const int64_t first = t0 == 0 ? -(int64_t)(W - 1) : t0;      // the first gradient that is this run's
        float win[W][kV], da[W][kV];        // da[j]: of the token j before the current one
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int v = 0; v < kV; ++v) da[j][v] = 0.f;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) P::unpack(in.at(t0 - (W - 1) + j), win[j + 1]);
        for (int64_t t = t0; t < t1 + W - 1; t += kBatch) {
            R xr[kBatch], gr[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool live = t + i < p.T && t + i < t1 + W - 1;
                xr[i] = live ? in.at(t + i) : R{};
                gr[i] = live ? *reinterpret_cast<const R *>(dyp + (t + i) * p.dy_t) : R{};
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (t + i >= t1 + W - 1) break;
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int v = 0; v < kV; ++v) win[j][v] = win[j + 1][v];
#pragma unroll
                for (int j = W - 1; j > 0; --j)
#pragma unroll
                    for (int v = 0; v < kV; ++v) da[j][v] = da[j - 1][v];
                P::unpack(xr[i], win[W - 1]);
                P::unpack(gr[i], da[0]);
                if (t + i < p.T) {
#pragma unroll
                    for (int v = 0; v < kV; ++v) {
                        float a = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) a = fmaf(w[j][v], win[j][v], a);
                        da[0][v] *= act_grad<T>(a, p.act);
                    }
                    if (t + i < t1) {
#pragma unroll
                        for (int v = 0; v < kV; ++v) {
                            db[v] += da[0][v];
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][v] = fmaf(da[0][v], win[j][v], dw[j][v]);
                        }
                    }
                }
                const int64_t at = t + i - (W - 1);       // the token whose gradient is complete
                if (at < first) continue;
                T *out = at >= 0 ? dx + at * p.C : ds0 ? ds0 + (at + W - 1) * p.C : nullptr;
                if (!out) continue;
                float g[kV];
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    g[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) g[v] = fmaf(w[j][v], da[j][v], g[v]);
                }
                if (dsT && at >= keep) {
                    float e[kV];
                    P::unpack(*reinterpret_cast<const R *>(dsT + (at - keep) * p.C), e);
#pragma unroll
                    for (int v = 0; v < kV; ++v) g[v] += e[v];
                }
                *reinterpret_cast<R *>(out) = P::pack(g);
            }
        }
    }
    if (!part) return;
    // the runs of the CTA are added in their order
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < kV; ++v) sums[threadIdx.x][v] = j < W ? dw[j < W ? j : 0][v] : db[v];
        __syncthreads();
        for (int k = threadIdx.x; k < pl.lanes * kV; k += kThreads) {
            const int64_t ch = (int64_t)blockIdx.y * pl.lanes * kV + k;
            if (ch >= p.C) continue;
            float s = 0.f;
            for (int r = 0; r < rows; ++r) s += sums[r * pl.lanes + k / kV][k % kV];
            part[((int64_t)blockIdx.x * (W + 1) + j) * p.C + ch] = s;
        }
    }
}

// dw and dbias from the parts, added in their order.
__global__ void __launch_bounds__(kThreads)
conv_sums_kernel(const float *part, int64_t parts, int64_t C, int W, float *dw, float *db) {
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= C * (W + 1)) return;
    const int64_t j = id / C, c = id - j * C;
    float s = 0.f;
    for (int64_t i = 0; i < parts; ++i) s += part[(i * (W + 1) + j) * C + c];
    if (j < W) {
        if (dw) dw[c * W + j] = s;
    } else if (db) {
        db[c] = s;
    }
}

// One token of each row on the pages of a pool. A thread has all of a channel vector's page.
template <typename T, int kV, int W>
__global__ void __launch_bounds__(128)
conv_step_kernel(const __grid_constant__ ConvProblem p, unsigned int *err) {
    using P = Pack<T, kV>;
    using R = typename P::raw;
    const int64_t nv = p.C / kV, id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t r = id / nv, c = (id - r * nv) * kV;
    if (r >= p.B) return;
    const int64_t slot = p.slots ? p.slots[r] : r;
    T *yp = static_cast<T *>(p.y) + r * p.C + c;
    float a[kV];
    if (slot < 0 || slot >= p.P) {      // an empty row
        if (slot >= p.P && c == 0) atomicOr(err, kDevErrPages);
#pragma unroll
        for (int v = 0; v < kV; ++v) a[v] = 0.f;
        *reinterpret_cast<R *>(yp) = P::pack(a);
        return;
    }
    T *sp = static_cast<T *>(p.S) + slot * (W - 1) * p.C + c;
    R raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const R *>(sp + j * p.C);
    raw[W - 1] = *reinterpret_cast<const R *>(static_cast<const T *>(p.x) + r * p.x_b + c);
    float w[W][kV];
    load_weights<T, kV, W>(p, c, w, a);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float x[kV];
        P::unpack(raw[j], x);
#pragma unroll
        for (int v = 0; v < kV; ++v) a[v] = fmaf(w[j][v], x[v], a[v]);
        if (j > 0) *reinterpret_cast<R *>(sp + (j - 1) * p.C) = raw[j];
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) a[v] = act_of<T>(a[v], p.act);
    *reinterpret_cast<R *>(yp) = P::pack(a);
}

bool on16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

// Whether rows of kV channels at a time are on 16 bytes everywhere.
bool vectors(const ConvProblem &p, int v) {
    const int es = p.io == 0 ? 2 : 4;
    return p.C % v == 0 && on16(p.x) && p.x_b * es % 16 == 0 && p.x_t * es % 16 == 0 &&
           (!p.dy || (on16(p.dy) && p.dy_b * es % 16 == 0 && p.dy_t * es % 16 == 0));
}

ConvPlan conv_plan(const ConvProblem &p, int v, int num_sms, int most) {
    ConvPlan pl;
    const int64_t nv = p.C / v;
    pl.lanes = 1;
    while (pl.lanes < 32 && pl.lanes < nv) pl.lanes *= 2;
    // long runs read less twice, short ones give more threads: the longest with four CTAs to an SM
    for (pl.run = most; pl.run > 8; pl.run /= 2)
        if (p.B * ((p.T + pl.run - 1) / pl.run) * nv >= (int64_t)4 * num_sms * kThreads) break;
    pl.runs = (p.T + pl.run - 1) / pl.run;
    return pl;
}
dim3 conv_grid(const ConvProblem &p, int v, const ConvPlan &pl) {
    const int rows = kThreads / pl.lanes;
    return dim3((unsigned)((p.B * pl.runs + rows - 1) / rows), (unsigned)((p.C / v + pl.lanes - 1) / pl.lanes));
}

// f.template run<T, kV, W>() for the problem's type, width and vectors.
template <typename T, int kV, typename F>
void by_width(int W, const F &f) {
    switch (W) {
        case 1: f.template run<T, kV, 1>(); break;
        case 2: f.template run<T, kV, 2>(); break;
        case 3: f.template run<T, kV, 3>(); break;
        case 4: f.template run<T, kV, 4>(); break;
        case 5: f.template run<T, kV, 5>(); break;
        case 6: f.template run<T, kV, 6>(); break;
        case 7: f.template run<T, kV, 7>(); break;
        default: f.template run<T, kV, 8>(); break;
    }
}
template <int kBf16, typename F>
void dispatch(const ConvProblem &p, const F &f) {
    if (p.io == 0) {
        if (vectors(p, kBf16)) by_width<__nv_bfloat16, kBf16>(p.W, f);
        else by_width<__nv_bfloat16, 1>(p.W, f);
    } else {
        if (vectors(p, 4)) by_width<float, 4>(p.W, f);
        else by_width<float, 1>(p.W, f);
    }
}

struct Fwd {
    const ConvProblem &p;
    int sms;
    cudaStream_t s;
    template <typename T, int kV, int W>
    void run() const {
        const ConvPlan pl = conv_plan(p, kV, sms, 64);
        conv_fwd_kernel<T, kV, W><<<conv_grid(p, kV, pl), kThreads, 0, s>>>(p, pl);
    }
};
struct Bwd {
    const ConvProblem &p;
    int sms;
    float *part;
    int64_t *parts;
    bool launch;
    cudaStream_t s;
    template <typename T, int kV, int W>
    void run() const {
        const ConvPlan pl = conv_plan(p, kV, sms, 64);
        const dim3 grid = conv_grid(p, kV, pl);
        *parts = grid.x;
        if (launch) conv_bwd_kernel<T, kV, W><<<grid, kThreads, 0, s>>>(p, pl, part);
    }
};
struct Step {
    const ConvProblem &p;
    unsigned int *err;
    cudaStream_t s;
    template <typename T, int kV, int W>
    void run() const {
        const int64_t n = p.B * (p.C / kV);
        conv_step_kernel<T, kV, W><<<(unsigned)((n + 127) / 128), 128, 0, s>>>(p, err);
    }
};

}  // namespace

cudaError_t launch_conv_fwd(const ConvProblem &p, int num_sms, cudaStream_t s) {
    dispatch<8>(p, Fwd{p, num_sms, s});
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

size_t conv_bwd_workspace_bytes(const ConvProblem &p, int num_sms) {
    // whatever the alignment: the scalar plan has at least as many parts as any other
    int64_t parts = 0;
    for (int v : {1, 4}) {
        if (p.C % v) continue;
        const ConvPlan pl = conv_plan(p, v, num_sms, 64);
        parts = std::max<int64_t>(parts, conv_grid(p, v, pl).x);
    }
    return (size_t)parts * (p.W + 1) * p.C * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvProblem &p, void *ws, int num_sms, cudaStream_t s) {
    int64_t parts = 0;
    float *part = p.dw || p.dbias ? static_cast<float *>(ws) : nullptr;
    dispatch<4>(p, Bwd{p, num_sms, part, &parts, true, s});
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (part) {
        const int64_t n = p.C * (p.W + 1);
        conv_sums_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(part, parts, p.C, p.W, p.dw,
                                                                                     p.dbias);
        e = cudaGetLastError();
        if (e == cudaSuccess) count_launches(1);
    }
    return e;
}

cudaError_t launch_conv_step(const ConvProblem &p, unsigned int *dev_err, cudaStream_t s) {
    dispatch<8>(p, Step{p, dev_err, s});
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
