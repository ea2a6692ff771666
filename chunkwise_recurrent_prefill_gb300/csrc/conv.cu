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
#include "launch.h"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kBwdCtas = 2;         // CTAs of the backward kernel to an SM

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

// kV values as pairs (of one value: its second is not used).
template <int kV>
using Pairs = float2[(kV + 1) / 2];
template <typename T, int kV>
__device__ __forceinline__ void unpack(typename Pack<T, kV>::raw r, Pairs<kV> &v) {
    float f[kV];
    Pack<T, kV>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < kV; i += 2) v[i / 2] = make_float2(f[i], i + 1 < kV ? f[i + 1 < kV ? i + 1 : 0] : 0.f);
}
template <typename T, int kV>
__device__ __forceinline__ typename Pack<T, kV>::raw pack(const Pairs<kV> &v) {
    float f[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) f[i] = i % 2 ? v[i / 2].y : v[i / 2].x;
    return Pack<T, kV>::pack(f);
}

template <int kV, int W>
__device__ __forceinline__ void load_weights(const ConvProblem &p, int64_t c, Pairs<kV> (&w)[W], Pairs<kV> &b) {
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        float *to[W + 1];
#pragma unroll
        for (int j = 0; j < W; ++j) to[j] = v % 2 ? &w[j][v / 2].y : &w[j][v / 2].x;
#pragma unroll
        for (int j = 0; j < W; ++j) *to[j] = __ldg(p.w + (c + v) * W + j);
        (v % 2 ? b[v / 2].y : b[v / 2].x) = p.bias ? __ldg(p.bias + c + v) : 0.f;
    }
    if (kV == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][0].y = 0.f;
        b[0].y = 0.f;
    }
}

// bias + w . win
template <int kV, int W>
__device__ __forceinline__ float2 weigh(const Pairs<kV> (&w)[W], const Pairs<kV> (&x)[W], float2 sum, int k) {
#pragma unroll
    for (int j = 0; j < W; ++j) sum = tc::fma2(w[j][k], x[j][k], sum);
    return sum;
}

// kSilu: the activation is known at compile time, else it is act.
template <typename T, bool kSilu>
__device__ __forceinline__ float2 act2(float2 a, int act) {
    if (kSilu) return tc::mul2(a, make_float2(logistic<T>(a.x), logistic<T>(a.y)));
    return make_float2(act_of<T>(a.x, act), act_of<T>(a.y, act));
}
template <typename T, bool kSilu>
__device__ __forceinline__ float2 grad2(float2 a, int act) {
    if (kSilu) {        // s (1 + a (1 - s))
        const float2 s = make_float2(logistic<T>(a.x), logistic<T>(a.y)), one = make_float2(1.f, 1.f);
        return tc::mul2(s, tc::fma2(a, tc::fma2(s, make_float2(-1.f, -1.f), one), one));
    }
    return make_float2(act_grad<T>(a.x, act), act_grad<T>(a.y, act));
}

template <typename T, int kV, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads)
conv_fwd_kernel(const __grid_constant__ ConvProblem p, const ConvPlan pl) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    // Tokens loaded at a time, while those before them are worked on: what is on its way bounds the rate (16 loads
    // of 8 bytes to a thread, 64 KB to an SM: 16384 x 4096 channels in 49 us, 5.5 TB/s, fp32 102; with 8 of them a seventh more).
    constexpr int kBatch = kV * sizeof(T) > 8 ? 8 : 16;
    using R = typename Pack<T, kV>::raw;
    const int lane = threadIdx.x % pl.lanes;
    const int64_t c = ((int64_t)blockIdx.y * pl.lanes + lane) * kV;
    const int64_t id = (int64_t)blockIdx.x * (kThreads / pl.lanes) + threadIdx.x / pl.lanes;
    const int64_t b = id / pl.runs;
    if (c >= p.C || b >= p.B) return;
    const int64_t t0 = (id - b * pl.runs) * pl.run;
    const int n = (int)min((int64_t)pl.run, p.T - t0);
    const int64_t tail = b * (W - 1) * p.C + c;
    const Inputs<T, kV> in{static_cast<const T *>(p.x) + b * p.x_b + c,
                           p.s0 ? static_cast<const T *>(p.s0) + tail : nullptr, p.x_t, p.C, W};
    const T *xp = in.x + t0 * p.x_t;
    T *yp = static_cast<T *>(p.y) + (b * p.T + t0) * p.C + c;
    R raw[kBatch] = {};
    auto load = [&](int i0) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i0 + i < n) raw[i] = *reinterpret_cast<const R *>(xp + i * p.x_t);
        xp += kBatch * p.x_t;
    };
    load(0);
    Pairs<kV> w[W], bias, win[W];       // win[j]: the input j - (W - 1) tokens from the current one
    load_weights<kV, W>(p, c, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) unpack<T, kV>(in.at(t0 - (W - 1) + j), win[j + 1]);
    for (int i0 = 0; i0 < n; i0 += kBatch) {
        R cur[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) cur[i] = raw[i];
        load(i0 + kBatch);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int k = 0; k < (kV + 1) / 2; ++k) win[j][k] = win[j + 1][k];
            unpack<T, kV>(cur[i], win[W - 1]);
            Pairs<kV> a;
#pragma unroll
            for (int k = 0; k < (kV + 1) / 2; ++k) a[k] = act2<T, kSilu>(weigh<kV, W>(w, win, bias[k], k), p.act);
            if (i0 + i < n) *reinterpret_cast<R *>(yp + i * p.C) = pack<T, kV>(a);
        }
        yp += kBatch * p.C;
    }
    if (p.sT && t0 + n == p.T) {        // the last run leaves the last inputs
        T *sT = static_cast<T *>(p.sT) + tail;
        for (int j = 0; j < W - 1; ++j) *reinterpret_cast<R *>(sT + j * p.C) = in.at(p.T - (W - 1) + j);
    }
}

// Sums of a CTA's runs go to part[blockIdx.x][W + 1][C]: dw, then dbias.
template <typename T, int kV, int W, bool kSilu>
__global__ void __launch_bounds__(kThreads, kBwdCtas)
conv_bwd_kernel(const __grid_constant__ ConvProblem p, const ConvPlan pl, float *part) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    constexpr int kBatch = 4, kP = (kV + 1) / 2;
    using R = typename Pack<T, kV>::raw;
    __shared__ float sums[W + 1][kThreads][kV];
    const int lane = threadIdx.x % pl.lanes, row = threadIdx.x / pl.lanes, rows = kThreads / pl.lanes;
    const int64_t c = ((int64_t)blockIdx.y * pl.lanes + lane) * kV;
    const int64_t id = (int64_t)blockIdx.x * rows + row;
    const int64_t b = id / pl.runs;
    Pairs<kV> dw[W], db;
#pragma unroll
    for (int k = 0; k < kP; ++k) {
        db[k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][k] = make_float2(0.f, 0.f);
    }
    if (c < p.C && b < p.B) {
        const int64_t t0 = (id - b * pl.runs) * pl.run;
        // own tokens, tokens read (the gradient of a token is complete W - 1 tokens later), and what the sequence has
        const int n = (int)min((int64_t)pl.run, p.T - t0), end = n + W - 1;
        const int have = (int)min((int64_t)end, p.T - t0);
        const int64_t tail = b * (W - 1) * p.C + c;
        const Inputs<T, kV> in{static_cast<const T *>(p.x) + b * p.x_b + c,
                               p.s0 ? static_cast<const T *>(p.s0) + tail : nullptr, p.x_t, p.C, W};
        const T *xp = in.x + t0 * p.x_t, *gp = static_cast<const T *>(p.dy) + b * p.dy_b + c + t0 * p.dy_t;
        const T *dsT = p.dsT ? static_cast<const T *>(p.dsT) + tail : nullptr;
        T *dx = static_cast<T *>(p.dx) + (b * p.T + t0 - (W - 1)) * p.C + c;     // of the token W - 1 before the current one
        T *ds0 = p.ds0 ? static_cast<T *>(p.ds0) + tail : nullptr;
        const int64_t keep = p.T - (W - 1) - t0;        // from here on a token is part of sT
        R xr[kBatch] = {}, gr[kBatch] = {};
        auto load = [&](int i0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (i0 + i < have) {
                    xr[i] = *reinterpret_cast<const R *>(xp + i * p.x_t);
                    gr[i] = *reinterpret_cast<const R *>(gp + i * p.dy_t);
                }
            }
            xp += kBatch * p.x_t;
            gp += kBatch * p.dy_t;
        };
        load(0);
        Pairs<kV> w[W], bias, win[W], da[W];            // da[j]: of the token j before the current one
        load_weights<kV, W>(p, c, w, bias);
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int k = 0; k < kP; ++k) da[j][k] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) unpack<T, kV>(in.at(t0 - (W - 1) + j), win[j + 1]);
        for (int i0 = 0; i0 < end; i0 += kBatch) {
            R xc[kBatch], gc[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                xc[i] = xr[i];
                gc[i] = gr[i];
            }
            load(i0 + kBatch);
            // batches whose tokens are all the run's own, and so are those whose gradients they complete
            const bool inner = i0 >= W - 1 && i0 + kBatch <= n && i0 + kBatch - W < keep;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int t = i0 + i, done = t - (W - 1);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int k = 0; k < kP; ++k) win[j][k] = win[j + 1][k];
#pragma unroll
                for (int j = W - 1; j > 0; --j)
#pragma unroll
                    for (int k = 0; k < kP; ++k) da[j][k] = da[j - 1][k];
                if (inner || t < have) {
                    unpack<T, kV>(xc[i], win[W - 1]);
                    unpack<T, kV>(gc[i], da[0]);
#pragma unroll
                    for (int k = 0; k < kP; ++k)
                        da[0][k] = tc::mul2(da[0][k], grad2<T, kSilu>(weigh<kV, W>(w, win, bias[k], k), p.act));
                } else {
#pragma unroll
                    for (int k = 0; k < kP; ++k) da[0][k] = win[W - 1][k] = make_float2(0.f, 0.f);
                }
                if (inner || t < n) {
#pragma unroll
                    for (int k = 0; k < kP; ++k) {
                        db[k] = tc::add2(db[k], da[0][k]);
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][k] = tc::fma2(da[0][k], win[j][k], dw[j][k]);
                    }
                }
                Pairs<kV> g;
#pragma unroll
                for (int k = 0; k < kP; ++k) g[k] = weigh<kV, W>(w, da, make_float2(0.f, 0.f), k);
                if (inner) {
                    *reinterpret_cast<R *>(dx + i * p.C) = pack<T, kV>(g);
                } else if (t < end && (done >= 0 || t0 == 0)) {
                    T *out = done >= 0 ? dx + i * p.C : ds0 ? ds0 + t * p.C : nullptr;
                    if (dsT && done >= keep) {
                        Pairs<kV> e;
                        unpack<T, kV>(*reinterpret_cast<const R *>(dsT + (done - keep) * p.C), e);
#pragma unroll
                        for (int k = 0; k < kP; ++k) g[k] = tc::add2(g[k], e[k]);
                    }
                    if (out) *reinterpret_cast<R *>(out) = pack<T, kV>(g);
                }
            }
            dx += kBatch * p.C;
        }
    }
    if (!part) return;
    // the runs of the CTA are added in their order
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const float2 s = j < W ? dw[j < W ? j : 0][v / 2] : db[v / 2];
            sums[j][threadIdx.x][v] = v % 2 ? s.y : s.x;
        }
    __syncthreads();
    const int tile = pl.lanes * kV;
    for (int k = threadIdx.x; k < tile * (W + 1); k += kThreads) {
        const int j = k / tile, i = k - j * tile;
        const int64_t ch = (int64_t)blockIdx.y * tile + i;
        if (ch >= p.C) continue;
        float s = 0.f;
        for (int r = 0; r < rows; ++r) s += sums[j][r * pl.lanes + i / kV][i % kV];
        part[((int64_t)blockIdx.x * (W + 1) + j) * p.C + ch] = s;
    }
}

// dw and dbias from the parts, added in their order.
__global__ void __launch_bounds__(kThreads)
conv_sums_kernel(const float *part, int64_t parts, int64_t C, int W, float *dw, float *db) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (id >= C * (W + 1)) return;
    const int64_t j = id / C, c = id - j * C;
    float s = 0.f;
#pragma unroll 8
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
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    using R = typename Pack<T, kV>::raw;
    const int64_t nv = p.C / kV, id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t r = id / nv, c = (id - r * nv) * kV;
    if (r >= p.B) return;
    const int64_t slot = p.slots ? p.slots[r] : r;
    T *yp = static_cast<T *>(p.y) + r * p.C + c;
    if (slot < 0 || slot >= p.P) {      // an empty row
        if (slot >= p.P && c == 0) atomicOr(err, kDevErrPages);
        *reinterpret_cast<R *>(yp) = R{};
        return;
    }
    T *sp = static_cast<T *>(p.S) + slot * (W - 1) * p.C + c;
    R raw[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j] = *reinterpret_cast<const R *>(sp + j * p.C);
    raw[W - 1] = *reinterpret_cast<const R *>(static_cast<const T *>(p.x) + r * p.x_b + c);
    Pairs<kV> w[W], bias, x[W];
    load_weights<kV, W>(p, c, w, bias);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        unpack<T, kV>(raw[j], x[j]);
        if (j > 0) *reinterpret_cast<R *>(sp + (j - 1) * p.C) = raw[j];
    }
    Pairs<kV> a;
#pragma unroll
    for (int k = 0; k < (kV + 1) / 2; ++k) a[k] = act2<T, false>(weigh<kV, W>(w, x, bias[k], k), p.act);
    *reinterpret_cast<R *>(yp) = pack<T, kV>(a);
}

// Whether rows are on whole vectors of v channels everywhere (what is contiguous starts on 16 bytes).
// Others go channel by channel (8 x 2047 tokens, bf16: 2044 channels 28.7 us and 48.1 for the gradients, 2045 39.5 and 122.6).
bool vectors(const ConvProblem &p, int v) {
    const uintptr_t bytes = v * (p.io == 0 ? 2 : 4);
    auto on = [&](const void *q, int64_t sb, int64_t st) {
        return reinterpret_cast<uintptr_t>(q) % bytes == 0 && sb % v == 0 && st % v == 0;
    };
    return p.C % v == 0 && on(p.x, p.x_b, p.x_t) && (!p.dy || on(p.dy, p.dy_b, p.dy_t));
}

// Short runs read more inputs twice, long ones leave SMs without work at the end. Forward: 64 tokens, or fewer until
// there are two CTAs to an SM (16384 x 4096 channels: 52 us with runs of 64, 58 with 32, 56 with 136). Backward,
// where a run reads W - 1 tokens of two tensors twice: as long as one round of resident CTAs allows (8 x 2047 x
// 2048 channels: 54 us with runs of 112, 68 with 64); but no more than 256, beyond which the rows in flight lie
// too far apart (16384 x 4096: 130 us with runs of 864, 111 with 64).
ConvPlan conv_plan(const ConvProblem &p, int v, int num_sms, bool backward) {
    ConvPlan pl;
    const int64_t nv = p.C / v;
    pl.lanes = 1;
    while (pl.lanes < 32 && pl.lanes < nv) pl.lanes *= 2;
    const int64_t tiles = (nv + pl.lanes - 1) / pl.lanes, rows = kThreads / pl.lanes;
    const int64_t slots = num_sms * kBwdCtas * rows / std::max<int64_t>(1, tiles * p.B);     // runs of a sequence
    const int64_t one_round = slots > 0 ? ((p.T + slots - 1) / slots + 7) / 8 * 8 : 1 << 30;
    if (backward && one_round <= 256) {
        pl.run = (int)std::max<int64_t>(8, one_round);
    } else {
        for (pl.run = 64; pl.run > 8; pl.run /= 2)
            if (p.B * ((p.T + pl.run - 1) / pl.run) * tiles >= 2 * num_sms * rows) break;
    }
    pl.runs = (p.T + pl.run - 1) / pl.run;
    return pl;
}
dim3 conv_grid(const ConvProblem &p, int v, const ConvPlan &pl) {
    const int rows = kThreads / pl.lanes;
    return dim3((unsigned)((p.B * pl.runs + rows - 1) / rows), (unsigned)((p.C / v + pl.lanes - 1) / pl.lanes));
}

// f.template run<T, kV, W>() for the problem's type, width and vectors.
template <typename T, int kV, typename F>
cudaError_t by_width(int W, const F &f) {
    switch (W) {
        case 1: return f.template run<T, kV, 1>();
        case 2: return f.template run<T, kV, 2>();
        case 3: return f.template run<T, kV, 3>();
        case 4: return f.template run<T, kV, 4>();
        case 5: return f.template run<T, kV, 5>();
        case 6: return f.template run<T, kV, 6>();
        case 7: return f.template run<T, kV, 7>();
        default: return f.template run<T, kV, 8>();
    }
}
template <int kBf16, int kF32, typename F>
cudaError_t dispatch(const ConvProblem &p, const F &f) {
    if (p.io == 0)
        return vectors(p, kBf16) ? by_width<__nv_bfloat16, kBf16>(p.W, f) : by_width<__nv_bfloat16, 1>(p.W, f);
    return vectors(p, kF32) ? by_width<float, kF32>(p.W, f) : by_width<float, 1>(p.W, f);
}

struct Fwd {
    const ConvProblem &p;
    int sms;
    cudaStream_t s;
    template <typename T, int kV, int W, bool kSilu>
    cudaError_t go() const {
        const ConvPlan pl = conv_plan(p, kV, sms, false);
        return launch(conv_fwd_kernel<T, kV, W, kSilu>, conv_grid(p, kV, pl), kThreads, 0, s, p, pl);
    }
    template <typename T, int kV, int W>
    cudaError_t run() const {
        return p.act == 1 ? go<T, kV, W, true>() : go<T, kV, W, false>();
    }
};
struct Bwd {
    const ConvProblem &p;
    int sms;
    float *part;
    int64_t *parts;
    cudaStream_t s;
    template <typename T, int kV, int W, bool kSilu>
    cudaError_t go() const {
        const ConvPlan pl = conv_plan(p, kV, sms, true);
        const dim3 grid = conv_grid(p, kV, pl);
        *parts = grid.x;
        return launch(conv_bwd_kernel<T, kV, W, kSilu>, grid, kThreads, 0, s, p, pl, part);
    }
    template <typename T, int kV, int W>
    cudaError_t run() const {
        return p.act == 1 ? go<T, kV, W, true>() : go<T, kV, W, false>();
    }
};
struct Step {
    const ConvProblem &p;
    unsigned int *err;
    cudaStream_t s;
    template <typename T, int kV, int W>
    cudaError_t run() const {
        const int64_t n = p.B * (p.C / kV);
        return launch(conv_step_kernel<T, kV, W>, dim3((unsigned)((n + 127) / 128)), 128, 0, s, p, err);
    }
};

}  // namespace

cudaError_t launch_conv_fwd(const ConvProblem &p, int num_sms, cudaStream_t s) {
    return dispatch<4, 4>(p, Fwd{p, num_sms, s});
}

size_t conv_bwd_workspace_bytes(const ConvProblem &p, int num_sms) {
    // whatever the alignment: the most parts of the plans for one channel and for four at a time
    int64_t parts = 0;
    for (int v : {1, 4}) {
        if (p.C % v) continue;
        const ConvPlan pl = conv_plan(p, v, num_sms, true);
        parts = std::max<int64_t>(parts, conv_grid(p, v, pl).x);
    }
    return (size_t)parts * (p.W + 1) * p.C * sizeof(float);
}

cudaError_t launch_conv_bwd(const ConvProblem &p, void *ws, int num_sms, cudaStream_t s) {
    int64_t parts = 0;
    float *part = p.dw || p.dbias ? static_cast<float *>(ws) : nullptr;
    const cudaError_t e = dispatch<4, 4>(p, Bwd{p, num_sms, part, &parts, s});
    if (e != cudaSuccess || !part) return e;
    const int64_t n = p.C * (p.W + 1);
    return launch(conv_sums_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), kThreads, 0, s, part, parts, p.C,
                  p.W, p.dw, p.dbias);
}

cudaError_t launch_conv_step(const ConvProblem &p, unsigned int *dev_err, cudaStream_t s) {
    return dispatch<8, 4>(p, Step{p, dev_err, s});
}

}  // namespace gla
