// Group norm with an activation, channels last (forward and backward), and an optional gate:
//     u = (x - mean) rstd w + b;   y = act(u), or u act(gate)
//     du = dy act'(u), or dy act(gate);  dgate = dy u act'(gate)
//     dx = rstd (du w - mean(du w) - xhat mean(du w xhat));  dw = sum du xhat;  db = sum du
//
// Every element is read once or twice and written once, so HBM bandwidth bounds all of it. Three
// routes, by shape:
//   rows : L = 1 and a group's channels fit the registers of a warp's lanes: one pass. A segment
//          of W lanes (a power of two) owns one group and walks over entries, so weights and the
//          channel sums of the backward pass stay in registers.
//   maps : L > 1 (or wide groups): the positions of an entry are cut into parts, one CTA each. Where
//          they are few (cluster_plan), the parts are a cluster and one kernel does it all; else a
//          first kernel leaves each part's statistics, a second one combines them and a third one
//          writes. The second reading of x comes from registers or from L2 when the tensor fits there.
//   plain: a CTA per group, element by element, and a CTA per channel for dw and db: groups of an odd
//          number of channels; strides or pointers that are not on a vector's bytes (16, or those of two
//          channels where a group is not whole 16-byte vectors); groups of more than 256 vectors (2048
//          bf16 or 1024 fp32 channels), or maps and groups of more than 128 vectors with more than
//          65535 entries.
// Means and variances: where a group is in registers, the mean and then the squared deviations from
// it. Else each thread takes the mean of its first vector as a pivot and sums the deviations from
// it and their squares; threads and parts are then merged as (count, mean, M2), in a fixed order.
// (M2 = sum of squares - (sum)^2 / n loses digits if the pivot is many standard deviations of the
// thread's own n values away from their mean. A value among them is sqrt(n) away at most, so that the
// worst case, a first value far off all others, leaves M2 good to n 2^-24.)
#include <cuda_bf16.h>

#include <atomic>

#include "gla_internal.h"
#include "norm.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float get(const float *p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// 16 bytes as pairs of floats (the arithmetic is in packed pairs throughout: with scalar
// instructions the rows kernels were bound by issue, at 40 instructions an element).
// Where a group's channels are not whole vectors of 16 bytes but an even number, a vector is two
// channels (a type of its own of the same size, so that pointers to it count elements).
struct BF16Pair {
    __nv_bfloat16 v;
};
struct F32Pair {
    float v;
};
template <typename T>
struct Vec;
template <>
struct Vec<F32Pair> {
    static constexpr int n = 2;
    using raw = uint2;
    using elem = float;
    static __device__ __forceinline__ void unpack(uint2 v, float2 (&f)[1]) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    }
    static __device__ __forceinline__ uint2 pack(const float2 (&f)[1]) {
        return make_uint2(__float_as_uint(f[0].x), __float_as_uint(f[0].y));
    }
};
template <>
struct Vec<BF16Pair> {
    static constexpr int n = 2;
    using raw = uint32_t;
    using elem = __nv_bfloat16;
    static __device__ __forceinline__ void unpack(uint32_t v, float2 (&f)[1]) { f[0] = tc::unpack_bf16(v); }
    static __device__ __forceinline__ uint32_t pack(const float2 (&f)[1]) { return tc::pack_bf16(f[0].x, f[0].y); }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    using raw = uint4;
    using elem = float;
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[2]) {
        f[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[2]) {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                          __float_as_uint(f[1].y));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    using raw = uint4;
    using elem = __nv_bfloat16;
    static __device__ __forceinline__ void unpack(uint4 v, float2 (&f)[4]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
        return make_uint4(tc::pack_bf16(f[0].x, f[0].y), tc::pack_bf16(f[1].x, f[1].y),
                          tc::pack_bf16(f[2].x, f[2].y), tc::pack_bf16(f[3].x, f[3].y));
    }
};
template <typename T>
using Raw = typename Vec<T>::raw;
using tc::add2;
using tc::fma2;
using tc::mul2;
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The logistic function 1 / (1 + 2^(-u log2 e)). Results that are rounded to bf16 take the hardware's
// approximate exponential and reciprocal (a few 2^-22 of the value, where u < 0 another 2^-23 |u|), flushing denormals: the exact
// functions, and even the fast ones with their care for denormals, made the kernels bound by issue.
template <typename T>
__device__ __forceinline__ float logistic(float u) {
    if (sizeof(T) == 4) return 1.f / (1.f + expf(-u));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename T>
__device__ __forceinline__ float act_of(float u, int act) {
    if (act == 1) return u * logistic<T>(u);
    if (act == 2) return 0.5f * u * (1.f + erff(u * 0.70710678f));
    return u;
}
template <typename T>
__device__ __forceinline__ float act_grad(float u, int act) {
    if (act == 1) {
        const float s = logistic<T>(u);
        return s * (1.f + u * (1.f - s));
    }
    if (act == 2)
        return 0.5f * (1.f + erff(u * 0.70710678f)) + u * expf(-0.5f * u * u) * 0.39894228f;
    return 1.f;
}

// Of pairs; kSilu: the activation is known at compile time, else it is act.
template <typename T, bool kSilu>
__device__ __forceinline__ float2 act_of2(float2 u, int act) {
    if (kSilu) return mul2(u, make_float2(logistic<T>(u.x), logistic<T>(u.y)));
    return make_float2(act_of<T>(u.x, act), act_of<T>(u.y, act));
}
// The activation and its derivative, from one logistic if it is silu.
template <typename T, bool kSilu>
__device__ __forceinline__ void act_and_grad2(float2 u, int act, float2 &a, float2 &g) {
    if (kSilu) {
        const float2 s = make_float2(logistic<T>(u.x), logistic<T>(u.y));
        a = mul2(u, s);
        g = fma2(a, fma2(s, both(-1.f), both(1.f)), s);     // s (1 + u (1 - s))
    } else {
        a = make_float2(act_of<T>(u.x, act), act_of<T>(u.y, act));
        g = make_float2(act_grad<T>(u.x, act), act_grad<T>(u.y, act));
    }
}

// Count, mean and sum of squared deviations of some values.
struct Stat {
    float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat &a, const Stat &b) {
    const float n = a.n + b.n;
    if (n == 0.f) return a;
    const float d = b.mean - a.mean, f = b.n / n, w = a.n * f;
    // (d w before d d: with an empty part w is zero, where d d may be infinite and 0 d d NaN)
    return Stat{n, fmaf(d, f, a.mean), fmaf(d * w, d, a.m2 + b.m2)};
}
__device__ __forceinline__ Stat merge_lanes(Stat s, int width) {
    for (int o = width >> 1; o > 0; o >>= 1) {
        // both partners form the same sum: the lower lane's part first
        const Stat t{__shfl_xor_sync(0xffffffffu, s.n, o), __shfl_xor_sync(0xffffffffu, s.mean, o),
                     __shfl_xor_sync(0xffffffffu, s.m2, o)};
        s = (threadIdx.x & o) ? merge(t, s) : merge(s, t);
    }
    return s;
}
__device__ __forceinline__ float sum_lanes(float v, int width) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);     // (width is the same in the warp)
    return v;
}
// A vector's weights from memory, or their default.
template <int N>
__device__ __forceinline__ void load_param(const float *p, int64_t c, float otherwise, float2 (&f)[N]) {
    if constexpr (N == 1) {
        f[0] = p ? *reinterpret_cast<const float2 *>(p + c) : make_float2(otherwise, otherwise);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float4 v = p ? *reinterpret_cast<const float4 *>(p + c + 2 * i)
                               : make_float4(otherwise, otherwise, otherwise, otherwise);
            f[i] = make_float2(v.x, v.y);
            f[i + 1] = make_float2(v.z, v.w);
        }
    }
}

// What the backward pass makes of one vector: xhat, du, and dgate in place of z.
template <typename T, bool kGate, bool kSilu, int N>
__device__ __forceinline__ void grad_vec(float2 (&x)[N], float2 (&dy)[N], float2 (&z)[N], const float2 (&w)[N],
                                         const float2 (&b)[N], float mean, float rstd, int act) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = mul2(add2(x[i], both(-mean)), both(rstd));
        const float2 u = fma2(x[i], w[i], b[i]);
        float2 a, g;
        act_and_grad2<T, kSilu>(kGate ? z[i] : u, act, a, g);
        if (kGate) {
            z[i] = mul2(mul2(dy[i], u), g);
            dy[i] = mul2(dy[i], a);
        } else {
            dy[i] = mul2(dy[i], g);
        }
    }
}

// ======================================================================= rows
// Lanes of a segment, vectors of a lane, and how segments share the work of a CTA.
struct RowPlan {
    int W;          // lanes per group
    int gpc;        // groups of a CTA (grid y covers all)
    int rp;         // entries a CTA handles at a time
    int cg;         // channels of a group
};

// A lane keeps VPL vectors of an entry (and those of the next one, on their way). Measured: 16384
// entries of 2048 gated bf16 channels in 16 groups (201 MB) 34 us in the kernel, 5.9 TB/s, 37 a call;
// with one vector to a lane (28 instructions an element) 47 a call.
template <typename T, int VPL, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_rows_fwd(const __grid_constant__ NormProblem p, const RowPlan r) {
    constexpr int V = Vec<T>::n;
    const int cg = r.cg, nv = cg / V;
    const int seg = threadIdx.x / r.W, lane = threadIdx.x % r.W;
    const int64_t g = (int64_t)blockIdx.y * r.gpc + seg % r.gpc;
    const int64_t n0 = (int64_t)blockIdx.x * r.rp + seg / r.gpc, step = (int64_t)gridDim.x * r.rp;
    const bool live = g < p.G && seg / r.gpc < r.rp;
    const int64_t c0 = (live ? g : 0) * cg;
    float2 w[VPL][V / 2], b[VPL][V / 2];
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
        const int v = lane + k * r.W;
        const int64_t c = c0 + (v < nv ? v : 0) * V;
        load_param(p.w, c, 1.f, w[k]);
        load_param(p.b, c, 0.f, b[k]);
    }
    const float inv = 1.f / (float)cg;
    Raw<T> xv[VPL], zv[VPL];
    const T *xp = static_cast<const T *>(p.x) + n0 * p.x_n + c0 + lane * V;
    const T *zp = static_cast<const T *>(p.gate) + (kGate ? n0 * p.gate_n + c0 + lane * V : 0);
    T *yp = static_cast<T *>(p.y) + n0 * p.C + c0 + lane * V;
    const int64_t xs = step * p.x_n, zs = step * p.gate_n, ys = step * p.C;
    auto load = [&](int64_t n) {
        const bool in = live && n < p.N;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            xv[k] = zv[k] = Raw<T>{};
            if (in && lane + k * r.W < nv) {
                xv[k] = *reinterpret_cast<const Raw<T> *>(xp + k * r.W * V);
                if (kGate) zv[k] = *reinterpret_cast<const Raw<T> *>(zp + k * r.W * V);
            }
        }
        xp += xs;
        if (kGate) zp += zs;
    };
    load(n0);
    // the whole warp walks together (the shuffles need every lane): rows past the end do nothing.
    // The next entry is loaded while this one is worked on.
    for (int64_t base = (int64_t)blockIdx.x * r.rp, n = n0; base < p.N; base += step, n += step, yp += ys) {
        float2 x[VPL][V / 2];
        Raw<T> zc[VPL];
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            Vec<T>::unpack(xv[k], x[k]);
            zc[k] = zv[k];
        }
        load(n + step);
        float2 sum = both(0.f), sq = both(0.f);     // (vectors past the group's are zeros)
#pragma unroll
        for (int k = 0; k < VPL; ++k)
#pragma unroll
            for (int i = 0; i < V / 2; ++i) sum = add2(sum, x[k][i]);
        const float mean = sum_lanes(sum.x + sum.y, r.W) * inv;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            float2 t = both(0.f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                x[k][i] = add2(x[k][i], both(-mean));
                t = fma2(x[k][i], x[k][i], t);
            }
            if (lane + k * r.W < nv) sq = add2(sq, t);
        }
        const float rstd = rsqrtf(fmaf(sum_lanes(sq.x + sq.y, r.W), inv, p.eps));
        if (!live || n >= p.N) continue;
        if (lane == 0) {
            if (p.mean) p.mean[n * p.G + g] = mean;
            if (p.rstd) p.rstd[n * p.G + g] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            if (lane + k * r.W >= nv) continue;
            float2 z[V / 2];
            if (kGate) Vec<T>::unpack(zc[k], z);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 u = fma2(mul2(x[k][i], both(rstd)), w[k][i], b[k][i]);
                x[k][i] = kGate ? mul2(u, act_of2<T, kSilu>(z[i], p.act)) : act_of2<T, kSilu>(u, p.act);
            }
            *reinterpret_cast<Raw<T> *>(yp + k * r.W * V) = Vec<T>::pack(x[k]);
        }
    }
}

// Partial channel sums: sums[part][0: dw, 1: db][C], part = blockIdx.x * rp + the entry slot.
// Measured: 8191 entries of 2048 gated bf16 channels (168 MB) 30 us, 5.6 TB/s, and 6 us for the sums
// of the channels' parts.
template <typename T, int VPL, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_rows_bwd(const __grid_constant__ NormProblem p, const RowPlan r, float *sums) {
    tc::pdl_launch_dependents();
    constexpr int V = Vec<T>::n;
    const int cg = r.cg, nv = cg / V;
    const int seg = threadIdx.x / r.W, lane = threadIdx.x % r.W;
    const int64_t g = (int64_t)blockIdx.y * r.gpc + seg % r.gpc;
    const int64_t n0 = (int64_t)blockIdx.x * r.rp + seg / r.gpc, step = (int64_t)gridDim.x * r.rp;
    const bool live = g < p.G && seg / r.gpc < r.rp;
    const int64_t c0 = (live ? g : 0) * cg;
    float2 w[VPL][V / 2], b[VPL][V / 2], dw[VPL][V / 2], db[VPL][V / 2];
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
        const int v = lane + k * r.W;
        const int64_t c = c0 + (v < nv ? v : 0) * V;
        load_param(p.w, c, 1.f, w[k]);
        load_param(p.b, c, 0.f, b[k]);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dw[k][i] = db[k][i] = both(0.f);
    }
    const float inv = 1.f / (float)cg;
    Raw<T> xv[VPL], dv[VPL], zv[VPL];
    float mean, rstd;
    const int64_t at0 = c0 + lane * V;
    const T *xp = static_cast<const T *>(p.x) + n0 * p.x_n + at0;
    const T *dp = static_cast<const T *>(p.dy) + n0 * p.dy_n + at0;
    const T *zp = static_cast<const T *>(p.gate) + (kGate ? n0 * p.gate_n + at0 : 0);
    const float *mp = p.mean + n0 * p.G + g, *rp = p.rstd + n0 * p.G + g;
    T *op = static_cast<T *>(p.dx) + n0 * p.C + at0;
    T *gp = static_cast<T *>(p.dgate) + (kGate ? n0 * p.C + at0 : 0);
    const int64_t xs = step * p.x_n, ds = step * p.dy_n, zs = step * p.gate_n, ms = step * p.G, os = step * p.C;
    auto load = [&](int64_t n) {
        const bool in = live && n < p.N;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            xv[k] = dv[k] = zv[k] = Raw<T>{};
            if (in && lane + k * r.W < nv) {
                xv[k] = *reinterpret_cast<const Raw<T> *>(xp + k * r.W * V);
                dv[k] = *reinterpret_cast<const Raw<T> *>(dp + k * r.W * V);
                if (kGate) zv[k] = *reinterpret_cast<const Raw<T> *>(zp + k * r.W * V);
            }
        }
        mean = in ? *mp : 0.f;
        rstd = in ? *rp : 0.f;
        xp += xs;
        dp += ds;
        if (kGate) zp += zs;
        mp += ms;
        rp += ms;
    };
    // (a lane with more than one vector has no registers for the next entry's)
    constexpr bool kAhead = VPL == 1;
    if (kAhead) load(n0);
    for (int64_t base = (int64_t)blockIdx.x * r.rp, n = n0; base < p.N;
         base += step, n += step, op += os, gp += kGate ? os : 0) {
        const bool in = live && n < p.N;
        if (!kAhead) load(n);
        Raw<T> xc[VPL], dc[VPL], zc[VPL];
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            xc[k] = xv[k];
            dc[k] = dv[k];
            zc[k] = zv[k];
        }
        const float mu = mean, rs = rstd;
        if (kAhead) load(n + step);
        float2 x[VPL][V / 2], d[VPL][V / 2], z[V / 2];
        float2 t1 = both(0.f), t2 = both(0.f);
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            const int v = lane + k * r.W;
            Vec<T>::unpack(xc[k], x[k]);
            Vec<T>::unpack(dc[k], d[k]);
            Vec<T>::unpack(zc[k], z);
            grad_vec<T, kGate, kSilu>(x[k], d[k], z, w[k], b[k], mu, rs, p.act);
            if (!in || v >= nv) continue;
            if (kGate) *reinterpret_cast<Raw<T> *>(gp + k * r.W * V) = Vec<T>::pack(z);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                dw[k][i] = fma2(d[k][i], x[k][i], dw[k][i]);
                db[k][i] = add2(db[k][i], d[k][i]);
                d[k][i] = mul2(d[k][i], w[k][i]);
                t1 = add2(t1, d[k][i]);
                t2 = fma2(d[k][i], x[k][i], t2);
            }
        }
        const float s1 = sum_lanes(t1.x + t1.y, r.W) * inv;
        const float s2 = sum_lanes(t2.x + t2.y, r.W) * inv;
        if (!in) continue;
#pragma unroll
        for (int k = 0; k < VPL; ++k) {
            if (lane + k * r.W >= nv) continue;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                x[k][i] = mul2(both(rs), fma2(x[k][i], both(-s2), add2(d[k][i], both(-s1))));
            *reinterpret_cast<Raw<T> *>(op + k * r.W * V) = Vec<T>::pack(x[k]);
        }
    }
    if (!sums || !live) return;
    float *sp = sums + ((int64_t)blockIdx.x * r.rp + seg / r.gpc) * 2 * p.C;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
        const int v = lane + k * r.W;
        if (v >= nv) continue;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            *reinterpret_cast<float2 *>(sp + c0 + v * V + 2 * i) = dw[k][i];
            *reinterpret_cast<float2 *>(sp + p.C + c0 + v * V + 2 * i) = db[k][i];
        }
    }
}

// ======================================================================= maps
// CTA = (part of the positions, block of whole groups, entry). Thread (tx, ty) owns one vector column
// and every ry-th position.
struct MapPlan {
    int parts;      // of an entry's positions
    int nvb;        // vector columns of a block (a multiple of a group's)
    int ry;         // positions at a time
    int nv, groups; // vector columns of a group, groups of a block
    int cols;       // vector columns of a row
    int len;        // positions of a part
};
struct MapPos {
    int tx, ty;
    int64_t n, l0, l1, v;   // v: vector column in the row
    bool live;
};
__device__ __forceinline__ MapPos map_pos(const NormProblem &p, const MapPlan &m) {
    MapPos q;
    q.tx = threadIdx.x % m.nvb;
    q.ty = threadIdx.x / m.nvb;
    q.n = blockIdx.z;
    q.l0 = (int64_t)m.len * blockIdx.x;
    q.l1 = min(q.l0 + m.len, p.L);
    q.v = (int64_t)blockIdx.y * m.nvb + q.tx;
    q.live = q.ty < m.ry && q.v < m.cols;
    return q;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_maps_stats(const __grid_constant__ NormProblem p, const MapPlan m, Stat *part) {
    constexpr int V = Vec<T>::n, kAhead = 4;
    tc::pdl_launch_dependents();
    __shared__ Stat sh[kThreads];
    const MapPos q = map_pos(p, m);
    Stat s{0.f, 0.f, 0.f};
    if (q.live && q.l0 + q.ty < q.l1) {
        const T *xp = static_cast<const T *>(p.x) + q.n * p.x_n + q.v * V;
        float pivot = 0.f;
        float2 t1 = both(0.f), t2 = both(0.f);
        const int64_t xs = m.ry * p.x_l;
        xp += (q.l0 + q.ty) * p.x_l;
        const int count = (int)((q.l1 - q.l0 - q.ty + m.ry - 1) / m.ry);
        for (int i0 = 0; i0 < count; i0 += kAhead) {
            Raw<T> xv[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (i0 + a < count) xv[a] = *reinterpret_cast<const Raw<T> *>(xp);
                xp += xs;
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (i0 + a < count) {
                    float2 f[V / 2];
                    Vec<T>::unpack(xv[a], f);
                    if (a == 0 && i0 == 0) {
                        float2 t = f[0];
#pragma unroll
                        for (int i = 1; i < V / 2; ++i) t = add2(t, f[i]);
                        pivot = (t.x + t.y) * (1.f / V);
                    }
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 d = add2(f[i], both(-pivot));
                        t1 = add2(t1, d);
                        t2 = fma2(d, d, t2);
                    }
                }
        }
        const float s1 = t1.x + t1.y, s2 = t2.x + t2.y, n = (float)count * V;
        const float d = s1 / n;
        s = Stat{n, pivot + d, fmaxf(fmaf(-s1, d, s2), 0.f)};
        if (!(s2 < INFINITY)) s.m2 = s2;    // infinity or NaN (which fmaxf would drop)
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    // a warp per group: its columns and position slots
    const int lane = threadIdx.x & 31, entries = m.nv * m.ry;
    for (int g = threadIdx.x >> 5; g < m.groups; g += kWarps) {
        Stat t{0.f, 0.f, 0.f};
        for (int e = lane; e < entries; e += 32) t = merge(t, sh[e / m.nv * m.nvb + g * m.nv + e % m.nv]);
        t = merge_lanes(t, 32);
        const int64_t gg = (int64_t)blockIdx.y * m.groups + g;
        if (lane == 0 && gg < p.G) part[((int64_t)q.n * p.G + gg) * m.parts + blockIdx.x] = t;
    }
}

// The parts' statistics of one group of one entry, a warp each -> mean and rstd (stat [N, G] for the
// next kernel, and the caller's). Combined here once: done by every CTA of the next kernel, it
// cost more than the whole of its other work (3 maps of 4095 x 512: 50 us).
__global__ void __launch_bounds__(kThreads)
norm_maps_combine(const __grid_constant__ NormProblem p, const MapPlan m, const Stat *part, float2 *stat) {
    tc::pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::pdl_wait_prerequisites();
    if (i >= p.N * p.G) return;
    Stat t{0.f, 0.f, 0.f};
    for (int e = lane; e < m.parts; e += 32) t = merge(t, part[i * m.parts + e]);
    t = merge_lanes(t, 32);
    if (lane != 0) return;
    const float rstd = 1.f / sqrtf(t.m2 / t.n + p.eps);
    stat[i] = make_float2(t.mean, rstd);
    if (p.mean) p.mean[i] = t.mean;
    if (p.rstd) p.rstd[i] = rstd;
}

template <typename T, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_maps_apply(const __grid_constant__ NormProblem p, const MapPlan m, const float2 *stat) {
    constexpr int V = Vec<T>::n, kAhead = 2;
    const MapPos q = map_pos(p, m);
    float2 w[V / 2], b[V / 2];
    const int64_t c = (q.live ? q.v : 0) * V;
    load_param(p.w, c, 1.f, w);
    load_param(p.b, c, 0.f, b);
    tc::pdl_wait_prerequisites();
    if (!q.live) return;
    const float2 st = stat[q.n * p.G + q.v / m.nv];
    const float mean = st.x, rstd = st.y;
    const T *xp = static_cast<const T *>(p.x) + q.n * p.x_n + c;
    const T *zp = static_cast<const T *>(p.gate) + (kGate ? q.n * p.gate_n + c : 0);
    T *yp = static_cast<T *>(p.y) + q.n * p.L * p.C + c;
    for (int64_t l = q.l0 + q.ty; l < q.l1; l += (int64_t)m.ry * kAhead) {
        Raw<T> xv[kAhead], zv[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (l + a * m.ry < q.l1) {
                xv[a] = *reinterpret_cast<const Raw<T> *>(xp + (l + a * m.ry) * p.x_l);
                if (kGate) zv[a] = *reinterpret_cast<const Raw<T> *>(zp + (l + a * m.ry) * p.gate_l);
            }
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (l + a * m.ry < q.l1) {
                float2 f[V / 2], z[V / 2];
                Vec<T>::unpack(xv[a], f);
                if (kGate) Vec<T>::unpack(zv[a], z);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    const float2 u = fma2(mul2(add2(f[i], both(-mean)), both(rstd)), w[i], b[i]);
                    f[i] = kGate ? mul2(u, act_of2<T, kSilu>(z[i], p.act)) : act_of2<T, kSilu>(u, p.act);
                }
                *reinterpret_cast<Raw<T> *>(yp + (l + a * m.ry) * p.C) = Vec<T>::pack(f);
            }
    }
}

// Sums of du w and du w xhat of each part and group -> part; channel sums -> sums[entry, part][2][C].
template <typename T, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_maps_bwd_stats(const __grid_constant__ NormProblem p, const MapPlan m, float2 *part, float *sums) {
    constexpr int V = Vec<T>::n;
    tc::pdl_launch_dependents();
    __shared__ float2 sh[kThreads];
    extern __shared__ __align__(16) float ch[];     // [threads][2 V + 4] channel sums of the position slots
    const MapPos q = map_pos(p, m);
    const int nv = m.nv;
    float2 dw[V / 2], db[V / 2], t1 = both(0.f), t2 = both(0.f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) dw[i] = db[i] = both(0.f);
    if (q.live) {
        const int64_t c = q.v * V, at = q.n * p.G + q.v / nv;
        float2 w[V / 2], b[V / 2];
        load_param(p.w, c, 1.f, w);
        load_param(p.b, c, 0.f, b);
        const float mean = p.mean[at], rstd = p.rstd[at];
        const T *xp = static_cast<const T *>(p.x) + q.n * p.x_n + c;
        const T *dp = static_cast<const T *>(p.dy) + q.n * p.dy_n + c;
        const T *zp = static_cast<const T *>(p.gate) + (kGate ? q.n * p.gate_n + c : 0);
#pragma unroll 2
        for (int64_t l = q.l0 + q.ty; l < q.l1; l += m.ry) {
            float2 x[V / 2], d[V / 2], z[V / 2];
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(xp + l * p.x_l), x);
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(dp + l * p.dy_l), d);
            if (kGate) Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(zp + l * p.gate_l), z);
            grad_vec<T, kGate, kSilu>(x, d, z, w, b, mean, rstd, p.act);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                dw[i] = fma2(d[i], x[i], dw[i]);
                db[i] = add2(db[i], d[i]);
                d[i] = mul2(d[i], w[i]);
                t1 = add2(t1, d[i]);
                t2 = fma2(d[i], x[i], t2);
            }
        }
    }
    sh[threadIdx.x] = make_float2(t1.x + t1.y, t2.x + t2.y);
    // (16 bytes more a thread, so that neighbours' sums do not share banks)
    float2 *mine = reinterpret_cast<float2 *>(ch + threadIdx.x * (2 * V + 4));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        mine[i] = dw[i];
        mine[V / 2 + i] = db[i];
    }
    __syncthreads();
    const int groups = m.groups, lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < groups; g += kWarps) {
        float a = 0.f, b = 0.f;
        for (int e = lane; e < nv * m.ry; e += 32) {
            const float2 t = sh[e / nv * m.nvb + g * nv + e % nv];
            a += t.x;
            b += t.y;
        }
        a = sum_lanes(a, 32);
        b = sum_lanes(b, 32);
        const int64_t gg = (int64_t)blockIdx.y * groups + g;
        if (lane == 0 && gg < p.G) part[((int64_t)q.n * p.G + gg) * m.parts + blockIdx.x] = make_float2(a, b);
    }
    if (!sums) return;
    float *sp = sums + ((int64_t)q.n * m.parts + blockIdx.x) * 2 * p.C;
    for (int e = threadIdx.x; e < m.nvb * 2 * V; e += kThreads) {
        const int tx = e / (2 * V), i = e % (2 * V);
        const int64_t c = ((int64_t)blockIdx.y * m.nvb + tx) * V + i % V;
        if (c >= p.C) continue;
        float t = 0.f;
        for (int y = 0; y < m.ry; ++y) t += ch[(y * m.nvb + tx) * (2 * V + 4) + i];
        sp[(i < V ? 0 : p.C) + c] = t;
    }
}

// The parts' sums of one group of one entry, a warp each -> their means.
__global__ void __launch_bounds__(kThreads)
norm_maps_bwd_combine(const __grid_constant__ NormProblem p, const MapPlan m, const float2 *part, float2 *mean) {
    tc::pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    tc::pdl_wait_prerequisites();
    if (i >= p.N * p.G) return;
    float a = 0.f, b = 0.f;
    for (int e = lane; e < m.parts; e += 32) {
        const float2 t = part[i * m.parts + e];
        a += t.x;
        b += t.y;
    }
    a = sum_lanes(a, 32);
    b = sum_lanes(b, 32);
    const float inv = 1.f / ((float)p.L * (float)(p.C / p.G));
    if (lane == 0) mean[i] = make_float2(a * inv, b * inv);
}

template <typename T, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_maps_bwd_apply(const __grid_constant__ NormProblem p, const MapPlan m, const float2 *means) {
    tc::pdl_launch_dependents();
    constexpr int V = Vec<T>::n;
    const MapPos q = map_pos(p, m);
    const int nv = m.nv;
    tc::pdl_wait_prerequisites();
    if (!q.live) return;
    const int64_t c = q.v * V, at = q.n * p.G + q.v / nv;
    float2 w[V / 2], b[V / 2];
    load_param(p.w, c, 1.f, w);
    load_param(p.b, c, 0.f, b);
    const float mean = p.mean[at], rstd = p.rstd[at], s1 = means[at].x, s2 = means[at].y;
    const T *xp = static_cast<const T *>(p.x) + q.n * p.x_n + c;
    const T *dp = static_cast<const T *>(p.dy) + q.n * p.dy_n + c;
    const T *zp = static_cast<const T *>(p.gate) + (kGate ? q.n * p.gate_n + c : 0);
    T *op = static_cast<T *>(p.dx) + q.n * p.L * p.C + c;
    T *gp = static_cast<T *>(p.dgate) + (kGate ? q.n * p.L * p.C + c : 0);
#pragma unroll 2
    for (int64_t l = q.l0 + q.ty; l < q.l1; l += m.ry) {
        float2 x[V / 2], d[V / 2], z[V / 2];
        Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(xp + l * p.x_l), x);
        Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(dp + l * p.dy_l), d);
        if (kGate) Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(zp + l * p.gate_l), z);
        grad_vec<T, kGate, kSilu>(x, d, z, w, b, mean, rstd, p.act);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            x[i] = mul2(both(rstd), fma2(x[i], both(-s2), fma2(d[i], w[i], both(-s1))));
        *reinterpret_cast<Raw<T> *>(op + l * p.C) = Vec<T>::pack(x);
        if (kGate) *reinterpret_cast<Raw<T> *>(gp + l * p.C) = Vec<T>::pack(z);
    }
}

// ======================================================================= maps of a cluster
// One kernel for maps that a cluster can hold: the CTAs of a cluster are the parts of one entry and
// block of groups, and read each other's statistics from shared memory. Blocks are as narrow as a
// 128-byte row allows, so that there are many; the last read of a peer is followed by an arrival
// that every CTA awaits before it leaves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ float peer(const float *p, int rank) {
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
constexpr int kMostGroups = 32;      // of a cluster's block
constexpr int kKeep = 16;

// The first kKeep vectors of a thread stay in registers from the statistics to the output; the rest
// is read again (from L2).
template <typename T, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads, 2)
norm_cluster_fwd(const __grid_constant__ NormProblem p, const MapPlan m) {
    constexpr int V = Vec<T>::n;
    __shared__ Stat sh[kThreads];
    __shared__ Stat part[kMostGroups];
    __shared__ float2 stat[kMostGroups];
    const MapPos q = map_pos(p, m);
    const int64_t c = (q.live ? q.v : 0) * V, first = q.l0 + q.ty;
    const int count = q.live && first < q.l1 ? (int)((q.l1 - first + m.ry - 1) / m.ry) : 0;
    const int64_t xs = m.ry * p.x_l, zs = m.ry * p.gate_l, ys = m.ry * p.C;
    const T *xp = static_cast<const T *>(p.x) + (count ? q.n * p.x_n + first * p.x_l + c : 0);
    Raw<T> xv[kKeep];
#pragma unroll
    for (int a = 0; a < kKeep; ++a)
        xv[a] = a < count ? *reinterpret_cast<const Raw<T> *>(xp + a * xs) : Raw<T>{};
    Stat s{0.f, 0.f, 0.f};
    if (count) {
        float2 f[V / 2], t1 = both(0.f), t2 = both(0.f);
        Vec<T>::unpack(xv[0], f);
        float2 t = f[0];
#pragma unroll
        for (int i = 1; i < V / 2; ++i) t = add2(t, f[i]);
        const float pivot = (t.x + t.y) * (1.f / V);
        auto add = [&](Raw<T> v) {
            Vec<T>::unpack(v, f);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 d = add2(f[i], both(-pivot));
                t1 = add2(t1, d);
                t2 = fma2(d, d, t2);
            }
        };
#pragma unroll
        for (int a = 0; a < kKeep; ++a)
            if (a < count) add(xv[a]);
#pragma unroll 4
        for (int a = kKeep; a < count; ++a) add(*reinterpret_cast<const Raw<T> *>(xp + a * xs));
        const float s1 = t1.x + t1.y, s2 = t2.x + t2.y, n = (float)count * V;
        const float d = s1 / n;
        s = Stat{n, pivot + d, fmaxf(fmaf(-s1, d, s2), 0.f)};
        if (!(s2 < INFINITY)) s.m2 = s2;    // infinity or NaN (which fmaxf would drop)
    }
    sh[threadIdx.x] = s;
    __syncthreads();
    const int lane = threadIdx.x & 31, entries = m.nv * m.ry;
    for (int g = threadIdx.x >> 5; g < m.groups; g += kWarps) {
        Stat t{0.f, 0.f, 0.f};
        for (int e = lane; e < entries; e += 32) t = merge(t, sh[e / m.nv * m.nvb + g * m.nv + e % m.nv]);
        t = merge_lanes(t, 32);
        if (lane == 0) part[g] = t;
    }
    cluster_arrive();
    float2 w[V / 2], b[V / 2];
    load_param(p.w, c, 1.f, w);
    load_param(p.b, c, 0.f, b);
    cluster_wait();
    for (int g = threadIdx.x >> 5; g < m.groups; g += kWarps) {
        Stat t{0.f, 0.f, 0.f};
        if (lane < m.parts) t = Stat{peer(&part[g].n, lane), peer(&part[g].mean, lane), peer(&part[g].m2, lane)};
        t = merge_lanes(t, 16);
        const float rstd = 1.f / sqrtf(t.m2 / t.n + p.eps);
        const int64_t gg = (int64_t)blockIdx.y * m.groups + g;
        if (lane != 0) continue;
        stat[g] = make_float2(t.mean, rstd);
        if (blockIdx.x != 0 || gg >= p.G) continue;
        if (p.mean) p.mean[q.n * p.G + gg] = t.mean;
        if (p.rstd) p.rstd[q.n * p.G + gg] = rstd;
    }
    cluster_arrive();
    __syncthreads();
    if (count) {
        const float2 st = stat[q.tx / m.nv];
        const T *zp = static_cast<const T *>(p.gate) + (kGate ? q.n * p.gate_n + first * p.gate_l + c : 0);
        T *yp = static_cast<T *>(p.y) + (q.n * p.L + first) * p.C + c;
        auto write = [&](Raw<T> v, int a) {
            float2 f[V / 2], z[V / 2];
            Vec<T>::unpack(v, f);
            if (kGate) Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(zp + a * zs), z);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 u = fma2(mul2(add2(f[i], both(-st.x)), both(st.y)), w[i], b[i]);
                f[i] = kGate ? mul2(u, act_of2<T, kSilu>(z[i], p.act)) : act_of2<T, kSilu>(u, p.act);
            }
            *reinterpret_cast<Raw<T> *>(yp + a * ys) = Vec<T>::pack(f);
        };
#pragma unroll
        for (int a = 0; a < kKeep; ++a)
            if (a < count) write(xv[a], a);
#pragma unroll 2
        for (int a = kKeep; a < count; ++a) write(*reinterpret_cast<const Raw<T> *>(xp + a * xs), a);
    }
    cluster_wait();
}

// sums: [N][2][C] where there are several entries; for one, dw and db come from here.
template <typename T, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
norm_cluster_bwd(const __grid_constant__ NormProblem p, const MapPlan m, float *sums) {
    tc::pdl_launch_dependents();
    constexpr int V = Vec<T>::n;
    __shared__ float2 sh[kThreads];
    __shared__ float2 part[kMostGroups], means[kMostGroups];
    extern __shared__ __align__(16) float ch[];     // [threads][2 V + 4] channel sums of the position slots
    float *cta = ch + kThreads * (2 * V + 4);       // [nvb][2 V], those of the CTA
    const MapPos q = map_pos(p, m);
    const int nv = m.nv, lane = threadIdx.x & 31;
    const int64_t c = (q.live ? q.v : 0) * V, first = q.l0 + q.ty;
    const int count = q.live && first < q.l1 ? (int)((q.l1 - first + m.ry - 1) / m.ry) : 0;
    const T *xp = static_cast<const T *>(p.x) + (count ? q.n * p.x_n + first * p.x_l + c : 0);
    const T *dp = static_cast<const T *>(p.dy) + (count ? q.n * p.dy_n + first * p.dy_l + c : 0);
    const T *zp = static_cast<const T *>(p.gate) + (kGate && count ? q.n * p.gate_n + first * p.gate_l + c : 0);
    const int64_t xs = m.ry * p.x_l, ds = m.ry * p.dy_l, zs = m.ry * p.gate_l, os = m.ry * p.C;
    float2 w[V / 2], b[V / 2];
    load_param(p.w, c, 1.f, w);
    load_param(p.b, c, 0.f, b);
    const int64_t at = q.n * p.G + (q.live ? q.v / nv : 0);
    const float mean = p.mean[at], rstd = p.rstd[at];
    {
        float2 dw[V / 2], db[V / 2], t1 = both(0.f), t2 = both(0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) dw[i] = db[i] = both(0.f);
#pragma unroll 2
        for (int a = 0; a < count; ++a) {
            float2 x[V / 2], d[V / 2], z[V / 2];
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(xp + a * xs), x);
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(dp + a * ds), d);
            if (kGate) Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(zp + a * zs), z);
            grad_vec<T, kGate, kSilu>(x, d, z, w, b, mean, rstd, p.act);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                dw[i] = fma2(d[i], x[i], dw[i]);
                db[i] = add2(db[i], d[i]);
                d[i] = mul2(d[i], w[i]);
                t1 = add2(t1, d[i]);
                t2 = fma2(d[i], x[i], t2);
            }
        }
        sh[threadIdx.x] = make_float2(t1.x + t1.y, t2.x + t2.y);
        float2 *mine = reinterpret_cast<float2 *>(ch + threadIdx.x * (2 * V + 4));
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            mine[i] = dw[i];
            mine[V / 2 + i] = db[i];
        }
    }
    __syncthreads();
    for (int g = threadIdx.x >> 5; g < m.groups; g += kWarps) {
        float u = 0.f, v = 0.f;
        for (int e = lane; e < nv * m.ry; e += 32) {
            const float2 t = sh[e / nv * m.nvb + g * nv + e % nv];
            u += t.x;
            v += t.y;
        }
        u = sum_lanes(u, 32);
        v = sum_lanes(v, 32);
        if (lane == 0) part[g] = make_float2(u, v);
    }
    const bool want = p.dw || p.db;
    if (want)
        for (int e = threadIdx.x; e < m.nvb * 2 * V; e += kThreads) {
            const int tx = e / (2 * V), i = e % (2 * V);
            float t = 0.f;
            for (int y = 0; y < m.ry; ++y) t += ch[(y * m.nvb + tx) * (2 * V + 4) + i];
            cta[e] = t;
        }
    cluster_arrive();
    cluster_wait();
    const float inv = 1.f / ((float)p.L * (float)(nv * V));
    for (int g = threadIdx.x >> 5; g < m.groups; g += kWarps) {
        float u = 0.f, v = 0.f;
        if (lane < m.parts) {
            u = peer(&part[g].x, lane);
            v = peer(&part[g].y, lane);
        }
        u = sum_lanes(u, 16);
        v = sum_lanes(v, 16);
        if (lane == 0) means[g] = make_float2(u * inv, v * inv);
    }
    if (want)       // the channels are shared out among the CTAs
        for (int e = blockIdx.x * kThreads + threadIdx.x; e < m.nvb * 2 * V; e += m.parts * kThreads) {
            const int i = e % (2 * V);
            const int64_t k = ((int64_t)blockIdx.y * m.nvb + e / (2 * V)) * V + i % V;
            if (k >= p.C) continue;
            float t = 0.f;
            for (int r = 0; r < m.parts; ++r) t += peer(&cta[e], r);
            float *to = sums ? sums + (q.n * 2 + (i >= V)) * p.C : i < V ? p.dw : p.db;
            if (to) to[k] = t;
        }
    cluster_arrive();
    __syncthreads();
    if (count) {
        const float2 mm = means[q.tx / nv];
        T *op = static_cast<T *>(p.dx) + (q.n * p.L + first) * p.C + c;
        T *gp = static_cast<T *>(p.dgate) + (kGate ? (q.n * p.L + first) * p.C + c : 0);
#pragma unroll 2
        for (int a = 0; a < count; ++a) {
            float2 x[V / 2], d[V / 2], z[V / 2];
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(xp + a * xs), x);
            Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(dp + a * ds), d);
            if (kGate) Vec<T>::unpack(*reinterpret_cast<const Raw<T> *>(zp + a * zs), z);
            grad_vec<T, kGate, kSilu>(x, d, z, w, b, mean, rstd, p.act);
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                x[i] = mul2(both(rstd), fma2(x[i], both(-mm.y), fma2(d[i], w[i], both(-mm.x))));
            *reinterpret_cast<Raw<T> *>(op + a * os) = Vec<T>::pack(x);
            if (kGate) *reinterpret_cast<Raw<T> *>(gp + a * os) = Vec<T>::pack(z);
        }
    }
    cluster_wait();
}

// dw, db: the partial sums added in order. Thread (channel, slice): 32 channels, 32 slices of parts.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
norm_sum_parts(const float *__restrict__ sums, int parts, int64_t C, float *dw, float *db) {
    __shared__ float sh[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t e = (int64_t)blockIdx.x * 32 + tx;      // 0 .. 2 C - 1
    float t = 0.f;
    tc::pdl_wait_prerequisites();
    if (e < 2 * C) {
#pragma unroll 8
        for (int i = ty; i < parts; i += 32) t += sums[i * 2 * C + e];
    }
    sh[ty][tx] = t;
    __syncthreads();
    t = sum_lanes(sh[tx][ty], 32);      // channel ty of this block, over the slices
    const int64_t c = (int64_t)blockIdx.x * 32 + ty;
    if (tx != 0 || c >= 2 * C) return;
    float *to = c < C ? dw : db;
    if (to) to[c < C ? c : c - C] = t;
}

// ======================================================================= plain
// Sum over the block, the same on every thread (a fixed order).
__device__ __forceinline__ float block_sum(float v, float *sh) {
    v = sum_lanes(v, 32);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int i = 0; i < kWarps; ++i) s += sh[i];
    return s;
}

// One CTA per (entry, group): mean, then the squared deviations from it, then the output.
template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_plain_fwd(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kWarps];
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
        if (p.gate)
            y = u * act_of<T>(get(static_cast<const T *>(p.gate) + n * p.gate_n + l * p.gate_l + c), p.act);
        else
            y = act_of<T>(u, p.act);
        put(static_cast<T *>(p.y) + (n * p.L + l) * p.C + c, y);
    }
}

struct Grad {
    float xh, du, dz;
};
template <typename T>
__device__ __forceinline__ Grad grad_at(const NormProblem &p, int64_t n, int64_t l, int64_t c, float mean,
                                        float rstd) {
    Grad r;
    r.xh = (get(static_cast<const T *>(p.x) + n * p.x_n + l * p.x_l + c) - mean) * rstd;
    const float u = fmaf(r.xh, p.w ? p.w[c] : 1.f, p.b ? p.b[c] : 0.f);
    const float dy = get(static_cast<const T *>(p.dy) + n * p.dy_n + l * p.dy_l + c);
    if (p.gate) {
        const float z = get(static_cast<const T *>(p.gate) + n * p.gate_n + l * p.gate_l + c);
        r.du = dy * act_of<T>(z, p.act);
        r.dz = dy * u * act_grad<T>(z, p.act);
    } else {
        r.du = dy * act_grad<T>(u, p.act);
        r.dz = 0.f;
    }
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
norm_plain_bwd(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kWarps];
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
__global__ void __launch_bounds__(kThreads)
norm_plain_dw(const __grid_constant__ NormProblem p) {
    __shared__ float sh[kWarps];
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

// ======================================================================= host
enum Route { kRows, kMaps, kPlain };
constexpr int kMostVpl = 4;

// Channels of a vector: 16 bytes, or two where a group is not whole vectors of 16 bytes.
int64_t vec_of(const NormProblem &p) {
    const int64_t full = p.io == 0 ? 8 : 4;
    return p.C / p.G % full == 0 ? full : 2;
}
int64_t elem_bytes(const NormProblem &p) { return p.io == 0 ? 2 : 4; }

// The route depends on the shape and strides, so that the workspace's size can be told before
// the pointers are known; pointers that are not on a vector's bytes fall back to plain at the launch.
Route route(const NormProblem &p, bool backward) {
    const int64_t V = vec_of(p), cg = p.C / p.G;
    if (cg % V != 0) return kPlain;
    int64_t strides = p.x_n | p.x_l;
    if (p.gate) strides |= p.gate_n | p.gate_l;
    if (backward) strides |= p.dy_n | p.dy_l;
    if (strides % V != 0) return kPlain;
    if (p.L == 1 && cg / V <= 32 * kMostVpl) return kRows;
    if (cg / V <= kThreads && p.N <= 65535) return kMaps;
    return kPlain;
}
bool aligned(const NormProblem &p) {
    const uintptr_t bytes = (uintptr_t)(vec_of(p) * elem_bytes(p)), params = vec_of(p) == 2 ? 8 : 16;
    return !((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.gate) |
              reinterpret_cast<uintptr_t>(p.dy)) & (bytes - 1)) &&
           !((reinterpret_cast<uintptr_t>(p.w) | reinterpret_cast<uintptr_t>(p.b)) & (params - 1));
}

// `per`: vectors of a lane, if the group has as many. Two forward (half the shuffles, and half of what
// a vector costs besides its arithmetic: 16384 x 2048 gated 47.8 -> 43.2 us), one backward, where the
// registers of two leave too few warps (8191 x 2048: 40 against 54 us).
RowPlan row_plan(const NormProblem &p, int per) {
    const int nv = (int)(p.C / p.G / vec_of(p));
    RowPlan r;
    r.cg = (int)(p.C / p.G);
    r.W = 1;
    while (r.W * per < nv && r.W < 32) r.W <<= 1;
    const int segs = kThreads / r.W;
    r.gpc = (int)min(p.G, (int64_t)segs);
    r.rp = segs / r.gpc;
    return r;
}
// About `per_sm` CTAs on every SM, each with at least one entry.
dim3 row_grid(const NormProblem &p, const RowPlan &r, int sms, int per_sm) {
    const int64_t gy = (p.G + r.gpc - 1) / r.gpc, most = (p.N + r.rp - 1) / r.rp;
    const int64_t gx = min(most, max((int64_t)1, (int64_t)sms * per_sm / gy));
    return dim3((unsigned)gx, (unsigned)gy);
}

MapPlan map_plan(const NormProblem &p, int sms) {
    const int64_t V = vec_of(p), nv = p.C / p.G / V;
    MapPlan m;
    m.nv = (int)nv;
    m.cols = (int)(p.C / V);
    m.nvb = (int)min((int64_t)m.cols, kThreads / nv * nv);
    m.groups = m.nvb / m.nv;
    m.ry = kThreads / m.nvb;
    // parts: about four CTAs an SM, of at least four rounds of positions
    const int64_t blocks = (p.C / V + m.nvb - 1) / m.nvb * p.N;
    const int64_t parts = max((int64_t)1, min((int64_t)sms * 4 / blocks, p.L / (4 * m.ry)));
    m.len = (int)((p.L + parts - 1) / parts);
    m.parts = (int)((p.L + m.len - 1) / m.len);
    return m;
}
dim3 map_grid(const NormProblem &p, const MapPlan &m) {
    return dim3((unsigned)m.parts, (unsigned)((p.C / vec_of(p) + m.nvb - 1) / m.nvb), (unsigned)p.N);
}

// The plan of a cluster of up to 16 CTAs, each thread with at least four rounds of positions if it
// is larger than one, and all clusters on the GPU at once; false where that leaves a thread more
// than kMostRounds (half of them backward). With two CTAs to an SM (the registers of 16 vectors), a
// cluster's placement within a GPC leaves room for 14 clusters of 16 or 36 of 8 (occupancy query on
// 152 SMs): 24 of 16 ran in two waves, 23 us against 19 for 24 of 8. Measured, clusters against three
// kernels, per call: 3 x 4095 x 512 20 us against 28, 1 x 16384 x 512 21 against 37, backward of
// 4 x 4096 x 512 26 against 33, 64 x 300 x 512 (single CTAs) 20.5 against 27; beyond the rule
// 300 x 64 x 512 (2400 CTAs) 68 against 26, 1 x 262144 x 64 211 against 31, backward of
// 1 x 16384 x 1024 79 against 59.
constexpr int kMostCluster = 16, kMostRounds = 32;
bool cluster_plan(const NormProblem &p, int sms, bool backward, MapPlan *out) {
    const int64_t V = vec_of(p), nv = p.C / p.G / V;
    MapPlan m;
    m.nv = (int)nv;
    m.cols = (int)(p.C / V);
    m.groups = (int)min(max((int64_t)1, 128 / (V * elem_bytes(p)) / nv), p.G);    // (128 bytes of a row)
    m.nvb = m.groups * m.nv;
    m.ry = kThreads / m.nvb;
    m.parts = 1;
    const int64_t blocks = (m.cols + m.nvb - 1) / m.nvb * p.N;
    auto fits = [&](int parts) { return blocks * parts * 10 <= (int64_t)sms * (parts > 8 ? 14 : 18); };
    // one CTA that keeps all its positions, if such CTAs fill the GPU once or twice over
    const bool one = blocks >= sms && blocks <= 4 * (int64_t)sms && p.L <= (int64_t)kKeep * m.ry;
    while (!one && m.parts < kMostCluster && (int64_t)m.parts * m.ry * 4 < p.L && fits(m.parts * 2)) m.parts *= 2;
    const int64_t len = (p.L + m.parts - 1) / m.parts;
    m.len = (int)len;
    *out = m;
    return (one || fits(m.parts)) && (len + m.ry - 1) / m.ry <= (backward ? kMostRounds / 2 : kMostRounds);
}
// Not the portable cluster size: asked for once for each kernel.
template <typename... A>
cudaError_t launch_cluster(void (*kernel)(A...), std::atomic<uint64_t> &done, dim3 grid, size_t smem, cudaStream_t s,
                           A... args) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(done.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute((const void *)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute cl[1];
    cl[0].id = cudaLaunchAttributeClusterDimension;
    cl[0].val.clusterDim.x = grid.x;
    cl[0].val.clusterDim.y = cl[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = cl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
constexpr int kBwdPerSm = 2;
dim3 combine_grid(const NormProblem &p) { return dim3((unsigned)((p.N * p.G + kWarps - 1) / kWarps)); }
size_t mean_bytes(const NormProblem &p) { return round256((size_t)(p.N * p.G) * sizeof(float2)); }

// Bytes of the parts' statistics, and parts of the channel sums.
size_t stat_bytes(const NormProblem &p, const MapPlan &m, bool backward) {
    return round256((size_t)(p.N * m.parts * p.G) * (backward ? sizeof(float2) : sizeof(Stat)));
}

template <typename... A>
cudaError_t launch_n(void (*kernel)(A...), dim3 grid, int threads, size_t smem, bool dependent, cudaStream_t s,
                     A... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e == cudaSuccess) count_launches(1);
    return e;
}
template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, size_t smem, bool dependent, cudaStream_t s, A... args) {
    return launch_n(kernel, grid, kThreads, smem, dependent, s, args...);
}

// As many CTAs as are resident at once: each walks over its entries with the next one on its way, and
// a second, partial round of CTAs costs up to a fifth (16384 x 2048 gated bf16, 2 to an SM: 38 us;
// with 3 to 8 to an SM 40 to 45).
template <auto kKernel>
cudaError_t launch_rows(const NormProblem &p, const RowPlan &r, int sms, cudaStream_t s) {
    static std::atomic<int> resident{0};
    int per_sm = resident.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kKernel, kThreads, 0);
        if (e != cudaSuccess) return e;
        per_sm = max(per_sm, 1);
        resident.store(per_sm, std::memory_order_relaxed);
    }
    return launch(kKernel, row_grid(p, r, sms, per_sm), 0, false, s, p, r);
}

template <typename T, bool kGate, bool kSilu>
cudaError_t run_fwd(const NormProblem &p, void *ws, int sms, cudaStream_t s) {
    const Route rt = aligned(p) ? route(p, false) : kPlain;
    if (rt == kRows) {
        const RowPlan r = row_plan(p, 2);
        const int vpl = (int)((p.C / p.G / Vec<T>::n + r.W - 1) / r.W);
        if (vpl == 1) return launch_rows<norm_rows_fwd<T, 1, kGate, kSilu>>(p, r, sms, s);
        if (vpl == 2) return launch_rows<norm_rows_fwd<T, 2, kGate, kSilu>>(p, r, sms, s);
        return launch_rows<norm_rows_fwd<T, 4, kGate, kSilu>>(p, r, sms, s);
    }
    if (rt == kMaps) {
        MapPlan m;
        if (cluster_plan(p, sms, false, &m)) {
            static std::atomic<uint64_t> done{0};
            return launch_cluster(norm_cluster_fwd<T, kGate, kSilu>, done, map_grid(p, m), 0, s, p, m);
        }
        m = map_plan(p, sms);
        Stat *part = static_cast<Stat *>(ws);
        float2 *stat = reinterpret_cast<float2 *>(static_cast<char *>(ws) + stat_bytes(p, m, false));
        cudaError_t e = launch(norm_maps_stats<T>, map_grid(p, m), 0, false, s, p, m, part);
        if (e != cudaSuccess) return e;
        e = launch(norm_maps_combine, combine_grid(p), 0, true, s, p, m, (const Stat *)part, stat);
        if (e != cudaSuccess) return e;
        return launch(norm_maps_apply<T, kGate, kSilu>, map_grid(p, m), 0, true, s, p, m, (const float2 *)stat);
    }
    return launch(norm_plain_fwd<typename Vec<T>::elem>, dim3((unsigned)(p.N * p.G)), 0, false, s, p);
}

template <typename T, bool kGate, bool kSilu>
cudaError_t run_bwd(const NormProblem &p, void *ws, int sms, cudaStream_t s) {
    const Route rt = aligned(p) ? route(p, true) : kPlain;
    const bool want = p.dw || p.db;
    cudaError_t e;
    if (rt == kPlain) {
        e = launch(norm_plain_bwd<typename Vec<T>::elem>, dim3((unsigned)(p.N * p.G)), 0, false, s, p);
        if (e != cudaSuccess || !want) return e;
        return launch(norm_plain_dw<typename Vec<T>::elem>, dim3((unsigned)p.C), 0, false, s, p);
    }
    float *sums = nullptr;
    int64_t parts;
    if (rt == kRows) {
        const RowPlan r = row_plan(p, 1);
        const int vpl = (int)((p.C / p.G / Vec<T>::n + r.W - 1) / r.W);
        const dim3 grid = row_grid(p, r, sms, kBwdPerSm);
        parts = (int64_t)grid.x * r.rp;
        if (want) sums = static_cast<float *>(ws);
        if (vpl == 1) e = launch(norm_rows_bwd<T, 1, kGate, kSilu>, grid, 0, false, s, p, r, sums);
        else if (vpl == 2) e = launch(norm_rows_bwd<T, 2, kGate, kSilu>, grid, 0, false, s, p, r, sums);
        else e = launch(norm_rows_bwd<T, 4, kGate, kSilu>, grid, 0, false, s, p, r, sums);
    } else {
        MapPlan m;
        if (cluster_plan(p, sms, true, &m)) {
            static std::atomic<uint64_t> done{0};
            if (want && p.N > 1) sums = static_cast<float *>(ws);
            const size_t smem = (size_t)(kThreads * (2 * Vec<T>::n + 4) + m.nvb * 2 * Vec<T>::n) * sizeof(float);
            e = launch_cluster(norm_cluster_bwd<T, kGate, kSilu>, done, map_grid(p, m), smem, s, p, m, sums);
            if (e != cudaSuccess || !sums) return e;
            return launch_n(norm_sum_parts, dim3((unsigned)((2 * p.C + 31) / 32)), kSumThreads, 0, true, s,
                            (const float *)sums, (int)p.N, p.C, p.dw, p.db);
        }
        m = map_plan(p, sms);
        float2 *part = static_cast<float2 *>(ws);
        parts = p.N * m.parts;
        float2 *means = reinterpret_cast<float2 *>(static_cast<char *>(ws) + stat_bytes(p, m, true));
        if (want) sums = reinterpret_cast<float *>(static_cast<char *>(ws) + stat_bytes(p, m, true) + mean_bytes(p));
        const size_t smem = (size_t)kThreads * (2 * Vec<T>::n + 4) * sizeof(float);
        e = launch(norm_maps_bwd_stats<T, kGate, kSilu>, map_grid(p, m), smem, false, s, p, m, part, sums);
        if (e != cudaSuccess) return e;
        e = launch(norm_maps_bwd_combine, combine_grid(p), 0, true, s, p, m, (const float2 *)part, means);
        if (e != cudaSuccess) return e;
        e = launch(norm_maps_bwd_apply<T, kGate, kSilu>, map_grid(p, m), 0, true, s, p, m, (const float2 *)means);
    }
    if (e != cudaSuccess || !want) return e;
    return launch_n(norm_sum_parts, dim3((unsigned)((2 * p.C + 31) / 32)), kSumThreads, 0, true, s,
                    (const float *)sums, (int)parts, p.C, p.dw, p.db);
}

}  // namespace

size_t norm_workspace_bytes(const NormProblem &p, bool backward, int num_sms) {
    // (a gate can only take the route to plain, which needs none)
    const Route rt = route(p, backward);
    if (rt == kPlain || (rt == kRows && !backward)) return 0;
    if (rt == kRows) {
        const RowPlan r = row_plan(p, 1);
        return (size_t)row_grid(p, r, num_sms, kBwdPerSm).x * r.rp * 2 * p.C * sizeof(float);
    }
    MapPlan m;
    if (cluster_plan(p, num_sms, backward, &m)) return backward && p.N > 1 ? (size_t)p.N * 2 * p.C * sizeof(float) : 0;
    m = map_plan(p, num_sms);
    return stat_bytes(p, m, backward) + mean_bytes(p) + (backward ? (size_t)(p.N * m.parts) * 2 * p.C * sizeof(float) : 0);
}

cudaError_t launch_norm_fwd(const NormProblem &p, void *ws, int num_sms, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (vec_of(p) == 2) {
        if (p.io == 0)
            return p.gate ? run_fwd<BF16Pair, true, false>(p, ws, num_sms, s)
                          : run_fwd<BF16Pair, false, false>(p, ws, num_sms, s);
        return p.gate ? run_fwd<F32Pair, true, false>(p, ws, num_sms, s)
                      : run_fwd<F32Pair, false, false>(p, ws, num_sms, s);
    }
    if (p.act == 1) {
        if (p.io == 0) return p.gate ? run_fwd<bf16, true, true>(p, ws, num_sms, s) : run_fwd<bf16, false, true>(p, ws, num_sms, s);
        return p.gate ? run_fwd<float, true, true>(p, ws, num_sms, s) : run_fwd<float, false, true>(p, ws, num_sms, s);
    }
    if (p.io == 0) return p.gate ? run_fwd<bf16, true, false>(p, ws, num_sms, s) : run_fwd<bf16, false, false>(p, ws, num_sms, s);
    return p.gate ? run_fwd<float, true, false>(p, ws, num_sms, s) : run_fwd<float, false, false>(p, ws, num_sms, s);
}

cudaError_t launch_norm_bwd(const NormProblem &p, void *ws, int num_sms, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if (vec_of(p) == 2) {
        if (p.io == 0)
            return p.gate ? run_bwd<BF16Pair, true, false>(p, ws, num_sms, s)
                          : run_bwd<BF16Pair, false, false>(p, ws, num_sms, s);
        return p.gate ? run_bwd<F32Pair, true, false>(p, ws, num_sms, s)
                      : run_bwd<F32Pair, false, false>(p, ws, num_sms, s);
    }
    if (p.act == 1) {
        if (p.io == 0) return p.gate ? run_bwd<bf16, true, true>(p, ws, num_sms, s) : run_bwd<bf16, false, true>(p, ws, num_sms, s);
        return p.gate ? run_bwd<float, true, true>(p, ws, num_sms, s) : run_bwd<float, false, true>(p, ws, num_sms, s);
    }
    if (p.io == 0) return p.gate ? run_bwd<bf16, true, false>(p, ws, num_sms, s) : run_bwd<bf16, false, false>(p, ws, num_sms, s);
    return p.gate ? run_bwd<float, true, false>(p, ws, num_sms, s) : run_bwd<float, false, false>(p, ws, num_sms, s);
}

}  // namespace gla
