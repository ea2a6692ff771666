// Linear attention with one decay per head, token by token in fp32 on CUDA cores: every dtype,
// head dimension and length, and the route of short bf16 sequences.
//
// The columns of the state are independent (out_t[z] needs S[:, z] alone), so a CTA owns 16 of
// them for one head and walks the tokens with its part of S in registers: thread (column, row
// group) holds RPT rows of one column. A token costs it RPT multiply-adds for the update and
// RPT for the read; nothing but the state's own multiply-add chain is serial, so eight tokens are
// unrolled, and their sums over the 8 row groups of a column take 7 shuffles together. x, y and z
// are staged as fp32 in shared memory TB tokens at a time, the next tile being loaded meanwhile.
#include <cuda_bf16.h>

#include "gla_internal.h"
#include "hda_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kCols = 16;          // state columns of a CTA
constexpr float kSlow = -0.5f;     // log-decays above it use l - 1 (see below)

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void store(float *dst, uint4 v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
        *reinterpret_cast<float4 *>(dst) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void store(float *dst, uint4 v) {
        *reinterpret_cast<uint4 *>(dst) = v;
    }
};

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// One tile of TB tokens on its way from global memory to shared memory: rows of W floats, of
// which the first `width` (a multiple of 8) exist. Rows past the end and columns past the width
// become zero.
template <typename T, int TB, int W>
struct Tile {
    static constexpr int V = Vec<T>::n;
    static constexpr int kVecs = TB * W / V;
    static constexpr int kPer = (kVecs + kThreads - 1) / kThreads;
    uint4 r[kPer];
    // base: this head's first element; row i of the walk is token (rev ? T - 1 - i : i)
    __device__ __forceinline__ void load(const T *base, int64_t ts, int64_t i0, int64_t Tn, bool rev,
                                         int width) {
#pragma unroll
        for (int a = 0; a < kPer; ++a) {
            const int e = threadIdx.x + a * kThreads;
            const int row = e / (W / V), col = (e % (W / V)) * V;
            const int64_t i = i0 + row;
            r[a] = make_uint4(0, 0, 0, 0);
            if (e < kVecs && i < Tn && col < width)
                r[a] = *reinterpret_cast<const uint4 *>(base + (rev ? Tn - 1 - i : i) * ts + col);
        }
    }
    __device__ __forceinline__ void store(float *dst) const {
#pragma unroll
        for (int a = 0; a < kPer; ++a) {
            const int e = threadIdx.x + a * kThreads;
            if (e < kVecs) Vec<T>::store(dst + (e / (W / V)) * W + (e % (W / V)) * V, r[a]);
        }
    }
};

template <typename T, int RPT, int TB>
__global__ void __launch_bounds__(kThreads)
hda_exact_kernel(const __grid_constant__ HdaProblem p) {
    constexpr int W = 8 * RPT;                 // rows of the state, padded
    __shared__ __align__(16) float xs[2][TB * W], ys[2][TB * W], zs[2][TB * kCols];
    __shared__ float os[TB][kCols];
    const HdaLin &m = p.lin[blockIdx.z];
    const int z0 = blockIdx.x * kCols;
    if (z0 >= m.Dz) return;
    const int64_t bh = blockIdx.y, b = bh / p.H, h = bh % p.H;
    const int lane = threadIdx.x & 31;
    // lanes 8 c .. 8 c + 7 of a warp are the row groups of one column; a row group's rows come
    // in fours, interleaved with the other groups', so that 16-byte reads of x and y meet no
    // bank twice
    const int rg = lane & 7, col = (threadIdx.x >> 5) * 4 + (lane >> 3);
    const bool in = z0 + col < m.Dz;
    auto row_of = [&](int k) { return (k >> 2) * 32 + rg * 4 + (k & 3); };
    auto head = [&](const HdaTensor &t) {
        return static_cast<const T *>(t.p) + b * t.b + (h / (p.H / t.heads)) * t.h;
    };
    const T *xp = head(m.x), *yp = head(m.y), *zp = head(m.z) + z0;
    const float g = p.decay[h];
    const bool rev = m.rev != 0;

    float s[RPT];
#pragma unroll
    for (int k = 0; k < RPT; ++k) {
        const int r = row_of(k), c = z0 + col;
        s[k] = 0.f;
        if (m.init && in && r < m.Dx)
            s[k] = m.init[bh * m.Dx * m.Dz + (m.init_t ? (int64_t)c * m.Dx + r
                                                       : (int64_t)r * m.Dz + c)];
    }

    // Reversed passes start from a state that already carries the step's decay: their first
    // token applies none. l s is formed as s + (l - 1) s for slow decays: l - 1 = expm1(g) is
    // known to 2^-24 of itself, so that a token's weight after n steps is off by 2^-24 n |g|,
    // not by 2^-24 n. Fast decays multiply by l itself (l = 0 leaves exactly the new token).
    const bool slow = g > kSlow;
    const float lam = expf(g), lm1 = expm1f(g);
    Tile<T, TB, W> tx, ty;
    Tile<T, TB, kCols> tz;
    const int zw = min(kCols, m.Dz - z0);
    tx.load(xp, m.x.t, 0, p.T, rev, m.Dx);
    ty.load(yp, m.y.t, 0, p.T, rev, m.Dx);
    tz.load(zp, m.z.t, 0, p.T, rev, zw);
    int buf = 0;
    for (int64_t i0 = 0; i0 < p.T; i0 += TB, buf ^= 1) {
        tx.store(xs[buf]);
        ty.store(ys[buf]);
        tz.store(zs[buf]);
        __syncthreads();
        if (i0 + TB < p.T) {
            tx.load(xp, m.x.t, i0 + TB, p.T, rev, m.Dx);
            ty.load(yp, m.y.t, i0 + TB, p.T, rev, m.Dx);
            tz.load(zp, m.z.t, i0 + TB, p.T, rev, zw);
        }
        const int nt = (int)min((int64_t)TB, p.T - i0);
        auto walk = [&](auto is_slow) {
#pragma unroll 1
            for (int i8 = 0; i8 < nt; i8 += 8) {
                float acc[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = 0.f;
                    if (i8 + i >= nt) continue;
                    const float zt = m.a_in * zs[buf][(i8 + i) * kCols + col];
                    const bool first = rev && i0 == 0 && i8 + i == 0;
                    const float f = first ? (is_slow ? 0.f : 1.f) : (is_slow ? lm1 : lam);
                    float part[2] = {0.f, 0.f};
#pragma unroll
                    for (int k4 = 0; k4 < RPT / 4; ++k4) {
                        const float4 y4 =
                            *reinterpret_cast<const float4 *>(&ys[buf][(i8 + i) * W + row_of(4 * k4)]);
                        const float4 x4 =
                            *reinterpret_cast<const float4 *>(&xs[buf][(i8 + i) * W + row_of(4 * k4)]);
                        const float yv[4] = {y4.x, y4.y, y4.z, y4.w}, xv[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &sk = s[4 * k4 + e];
                            sk = is_slow ? fmaf(f, sk, fmaf(yv[e], zt, sk)) : fmaf(f, sk, yv[e] * zt);
                            part[e & 1] = fmaf(xv[e], sk, part[e & 1]);
                        }
                    }
                    acc[i] = part[0] + part[1];
                }
                // sums over the 8 row groups, of 8 tokens at once: each step halves the tokens a lane
                // holds, and lane rg is left with token rg
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bool up = rg & 4;
                    const float keep = up ? acc[i + 4] : acc[i], give = up ? acc[i] : acc[i + 4];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool up = rg & 2;
                    const float keep = up ? acc[i + 2] : acc[i], give = up ? acc[i] : acc[i + 2];
                    acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
                }
                {
                    const bool up = rg & 1;
                    const float keep = up ? acc[1] : acc[0], give = up ? acc[0] : acc[1];
                    acc[0] = keep + __shfl_xor_sync(0xffffffffu, give, 1);
                }
                os[i8 + rg][col] = m.a_out * acc[0];
            }
        };
        if (slow) walk(std::true_type{});
        else walk(std::false_type{});
        __syncthreads();
        for (int e = threadIdx.x; e < nt * kCols; e += kThreads) {
            const int i = e / kCols, c = e % kCols;
            if (z0 + c >= m.Dz) continue;
            const int64_t t = rev ? p.T - 1 - (i0 + i) : i0 + i;
            const int64_t at = ((b * p.T + t) * p.H + h) * m.Dz + z0 + c;
            if (m.out_f32) static_cast<float *>(m.out)[at] = os[i][c];
            else put(static_cast<T *>(m.out) + at, os[i][c]);
        }
    }
    if (m.fin && in) {
#pragma unroll
        for (int k = 0; k < RPT; ++k) {
            const int r = row_of(k), c = z0 + col;
            float v = s[k];
            if (rev && p.T > 0) v = slow ? fmaf(lm1, v, v) : lam * v;
            if (r < m.Dx)
                m.fin[bh * m.Dx * m.Dz + (m.fin_t ? (int64_t)c * m.Dx + r
                                                  : (int64_t)r * m.Dz + c)] = v;
        }
    }
}

// Gradients of shared heads: the state heads' parts are added in fp32 in the order of the
// heads, and rounded once.
template <typename T>
__global__ void hda_share_kernel(HdaShare a, HdaShare b, HdaShare c, int64_t BT, int64_t H) {
    const HdaShare s = blockIdx.y == 0 ? a : blockIdx.y == 1 ? b : c;
    const int64_t n = BT * s.heads * (s.D / 4);
    const int rep = (int)(H / s.heads);
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t d4 = e % (s.D / 4), th = e / (s.D / 4);   // th = token * heads + head
        const float *ip = s.in + th * rep * s.D + d4 * 4;
        float4 v = *reinterpret_cast<const float4 *>(ip);
        for (int r = 1; r < rep; ++r) {
            const float4 w = *reinterpret_cast<const float4 *>(ip + (int64_t)r * s.D);
            v.x += w.x;
            v.y += w.y;
            v.z += w.z;
            v.w += w.w;
        }
        T *op = static_cast<T *>(s.out) + e * 4;
        put(op, v.x);
        put(op + 1, v.y);
        put(op + 2, v.z);
        put(op + 3, v.w);
    }
}

template <typename T>
cudaError_t run_exact(const HdaProblem &p, cudaStream_t s) {
    int dx = 0, dz = 0;
    for (int i = 0; i < p.n; ++i) {
        dx = max(dx, p.lin[i].Dx);
        dz = max(dz, p.lin[i].Dz);
    }
    // the batch entries are cut so that the grid's y dimension stays within its limit
    const int64_t most = 65535 / p.H > 0 ? 65535 / p.H : 1;
    for (int64_t b0 = 0; b0 < p.B; b0 += most) {
        HdaProblem c = p;
        c.B = min(most, p.B - b0);
        for (int i = 0; i < p.n; ++i) {
            HdaLin &m = c.lin[i];
            for (HdaTensor *t : {&m.x, &m.y, &m.z}) t->p = static_cast<const T *>(t->p) + b0 * t->b;
            const int64_t st = b0 * p.H * m.Dx * m.Dz, ot = b0 * p.T * p.H * m.Dz;
            if (m.init) m.init += st;
            if (m.fin) m.fin += st;
            m.out = static_cast<char *>(m.out) + ot * (m.out_f32 ? 4 : (int64_t)sizeof(T));
        }
        const dim3 grid((dz + kCols - 1) / kCols, (unsigned)(c.B * p.H), p.n);
        if (dx <= 64) hda_exact_kernel<T, 8, 16><<<grid, kThreads, 0, s>>>(c);
        else if (dx <= 128) hda_exact_kernel<T, 16, 16><<<grid, kThreads, 0, s>>>(c);
        else hda_exact_kernel<T, 32, 8><<<grid, kThreads, 0, s>>>(c);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_hda_exact(const HdaProblem &p, cudaStream_t s) {
    return p.io == 0 ? run_exact<__nv_bfloat16>(p, s) : run_exact<float>(p, s);
}

cudaError_t launch_hda_share(const HdaShare *parts, int n, int64_t BT, int64_t H, int io,
                             cudaStream_t s) {
    if (n == 0 || BT == 0) return cudaSuccess;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) most = max(most, BT * parts[i].heads * (parts[i].D / 4));
    const dim3 grid((unsigned)min((most + 255) / 256, (int64_t)152 * 8), n);
    const HdaShare b = parts[n > 1 ? 1 : 0], c = parts[n > 2 ? 2 : 0];
    if (io == 0) hda_share_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(parts[0], b, c, BT, H);
    else hda_share_kernel<float><<<grid, 256, 0, s>>>(parts[0], b, c, BT, H);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
