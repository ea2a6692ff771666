// Linear attention with one decay per head, token by token in fp32 on CUDA cores: every dtype,
// head dimension and length, and the route of short bf16 sequences.
//
// The columns of the state are independent (out_t[z] needs S[:, z] alone), so a CTA owns 16 NC of
// them for one head and walks the tokens with its part of S in registers: a thread holds RPT rows of
// NC columns (packed in pairs of rows), 8 threads the rows of a column. A token costs it two
// multiply-adds per element of S, or three where the decay is fast; with one column per thread the
// reads of x and y from shared memory take more than three times as long. Nothing but the state's own
// addition chain is serial. The sums over the 8 row groups are formed for 8 (token, column) pairs at
// once, in 7 shuffles. x, y and z are staged as fp32 in shared memory TB tokens at a time, the next
// tile being loaded meanwhile.
//
// A walk is serial, so where long sequences give the SMs few CTAs it is cut into segments: one kernel
// walks all but the last for their end states alone (from zero, but the first), a second one makes
// start states of them,
//     S(1) = E(0),  S(j + 1) = l^len S(j) + E(j),
// and a third one walks all segments for the outputs (one head of 16384 tokens: 2050 us -> 82).
#include <cuda_bf16.h>

#include "gla_internal.h"
#include "hda_internal.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr float kSlow = 0.5f;      // log-decays below it, of either sign, are applied by the tile (see below)

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void store(float *dst, uint4 v, float by = 1.f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = by * __uint_as_float(w[i] << 16);
            f[2 * i + 1] = by * __uint_as_float(w[i] & 0xffff0000u);
        }
        *reinterpret_cast<float4 *>(dst) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(f[4], f[5], f[6], f[7]);
    }
};
template <>
struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void store(float *dst, uint4 v, float by = 1.f) {
        *reinterpret_cast<float4 *>(dst) = make_float4(by * __uint_as_float(v.x), by * __uint_as_float(v.y),
                                                       by * __uint_as_float(v.z), by * __uint_as_float(v.w));
    }
};

__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
}

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
    __device__ __forceinline__ void load(const T *base, int64_t ts, int64_t i0, int64_t end, int64_t Tn,
                                         bool rev, int width) {
#pragma unroll
        for (int a = 0; a < kPer; ++a) {
            const int e = threadIdx.x + a * kThreads;
            const int row = e / (W / V), col = (e % (W / V)) * V;
            const int64_t i = i0 + row;
            r[a] = make_uint4(0, 0, 0, 0);
            if (e < kVecs && i < end && col < width)
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
    // each token times its factor
    __device__ __forceinline__ void store(float *dst, const float *by) const {
#pragma unroll
        for (int a = 0; a < kPer; ++a) {
            const int e = threadIdx.x + a * kThreads, row = e / (W / V);
            if (e < kVecs) Vec<T>::store(dst + row * W + (e % (W / V)) * V, r[a], by[row]);
        }
    }
};

struct Segs {
    int n, zblocks;         // segments, CTAs of a segment
    int64_t len;            // tokens of a segment
    float2 *E;              // end states: [map][head][segment 0 .. n - 2][CTA][pair][thread]
};

// kState: the segments' end states only.
template <typename T, int RPT, int NC, int TB, bool kState>
__global__ void __launch_bounds__(kThreads)
hda_exact_kernel(const __grid_constant__ HdaProblem p, const Segs sg) {
    constexpr int W = 8 * RPT;                 // rows of the state, padded
    constexpr int kCols = 16 * NC, G = 8 / NC; // columns of the CTA; tokens at a time
    __shared__ __align__(16) float xs[kState ? 1 : 2][kState ? 4 : TB * W], ys[2][TB * W], zs[2][TB * kCols];
    __shared__ float os[kState ? 1 : TB][kCols];
    __shared__ float pw[TB + 1], zf[2 * TB], of[TB];    // l^i; factors of z and of the outputs
    if (kState) tc::pdl_launch_dependents();
    const int li = blockIdx.z % p.n;
    const int64_t bh = (int64_t)(blockIdx.z / p.n) * gridDim.y + blockIdx.y, b = bh / p.H, h = bh % p.H;
    const HdaLin &m = p.lin[li];
    const int zb = blockIdx.x % sg.zblocks, seg = blockIdx.x / sg.zblocks, z0 = zb * kCols;
    if (z0 >= m.Dz || b >= p.B) return;
    const int64_t begin = seg * sg.len, end = min(begin + sg.len, p.T);
    const int lane = threadIdx.x & 31;
    // lanes 8 c .. 8 c + 7 of a warp are the row groups of NC columns; a row group's rows come
    // in fours, interleaved with the other groups', so that 16-byte reads of x and y meet no
    // bank twice
    const int rg = lane & 7, col = ((threadIdx.x >> 5) * 4 + (lane >> 3)) * NC;
    auto row_of = [&](int k) { return (k >> 2) * 32 + rg * 4 + (k & 3); };
    auto head = [&](const HdaTensor &t) {
        return static_cast<const T *>(t.p) + b * t.b + (h / (p.H / t.heads)) * t.h;
    };
    const T *xp = head(m.x), *yp = head(m.y), *zp = head(m.z) + z0;
    const float g = p.decay[h];
    const bool rev = m.rev != 0;

    float2 s[NC][RPT / 2];      // rows 2 k, 2 k + 1 of the thread's
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < RPT; ++k) {
            const int r = row_of(k), z = z0 + col + c;
            float v = 0.f;
            if (m.init && seg == 0 && z < m.Dz && r < m.Dx)
                v = m.init[bh * m.Dx * m.Dz + (m.init_t ? (int64_t)z * m.Dx + r : (int64_t)r * m.Dz + z)];
            (k & 1 ? s[c][k / 2].y : s[c][k / 2].x) = v;
        }
    constexpr int kPer = NC * RPT / 2;      // pairs of a thread
    float2 *E = sg.E + (((li * p.B * p.H + bh) * (sg.n - 1)) * sg.zblocks + zb) * (kPer * kThreads) +
                threadIdx.x;
    const int64_t e_seg = (int64_t)sg.zblocks * (kPer * kThreads);
    if (!kState && seg > 0) {
        tc::pdl_wait_prerequisites();
#pragma unroll
        for (int k = 0; k < kPer; ++k) s[k / (RPT / 2)][k % (RPT / 2)] = E[(seg - 1) * e_seg + k * kThreads];
    }

    // Reversed passes start from a state that already carries the step's decay: their first
    // token applies none. Slow decays are applied by the tile: within one the state is kept as it
    // will have decayed at the tile's end, S' = l^r S with r tokens left, so that S is multiplied once
    // in a tile, a token adds y (l^r z), and its output is l^-r (x S'). (l itself for every token would
    // be off by 2^-25 each time, always the same way; l S as S + (l - 1) S is NaN for an infinite S.)
    // Fast decays multiply by l itself (l = 0 leaves exactly the new token).
    const bool slow = fabsf(g) < kSlow;
    const float lam = expf(g);
    Tile<T, TB, W> tx, ty;
    Tile<T, TB, kCols> tz;
    const int zw = min(kCols, m.Dz - z0);
    if (!kState) tx.load(xp, m.x.t, begin, end, p.T, rev, m.Dx);
    ty.load(yp, m.y.t, begin, end, p.T, rev, m.Dx);
    tz.load(zp, m.z.t, begin, end, p.T, rev, zw);
    // Token i of a tile of nt is row i + TB - nt of the factors (rows past its end: any number).
    if (threadIdx.x < 2 * TB) {
        const int r = max(TB - 1 - (int)threadIdx.x, 0);
        zf[threadIdx.x] = m.a_in * (slow ? decay_pow(g, (float)r) : 1.f);
        if (threadIdx.x < TB) of[threadIdx.x] = m.a_out * (slow ? decay_pow(-g, (float)r) : 1.f);
        if (threadIdx.x <= TB) pw[threadIdx.x] = decay_pow(g, (float)threadIdx.x);
    }
    __syncthreads();
    int buf = 0;
    for (int64_t i0 = begin; i0 < end; i0 += TB, buf ^= 1) {
        const int nt = (int)min((int64_t)TB, end - i0);
        if (!kState) tx.store(xs[buf]);
        ty.store(ys[buf]);
        tz.store(zs[buf], zf + TB - nt);
        __syncthreads();
        if (i0 + TB < end) {
            if (!kState) tx.load(xp, m.x.t, i0 + TB, end, p.T, rev, m.Dx);
            ty.load(yp, m.y.t, i0 + TB, end, p.T, rev, m.Dx);
            tz.load(zp, m.z.t, i0 + TB, end, p.T, rev, zw);
        }
        if (slow) {
            const float f = pw[rev && i0 == 0 ? nt - 1 : nt];
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int k = 0; k < RPT / 2; ++k) s[c][k] = tc::mul2(make_float2(f, f), s[c][k]);
        }
        auto walk = [&](auto is_slow) {
#pragma unroll 1
            for (int i8 = 0; i8 < nt; i8 += G) {
                float acc[8];
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    // (no branch: the loads of later tokens are to be issued ahead. A token past the
                    // end is all zeros and applies no decay.)
                    float zt[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) zt[c] = zs[buf][(i8 + i) * kCols + col + c];
                    const bool none = i8 + i >= nt || (rev && i0 + i8 + i == 0);
                    const float f = none ? 1.f : lam;
                    const float2 ff = make_float2(f, f);
                    float2 part[NC];
#pragma unroll
                    for (int c = 0; c < NC; ++c) part[c] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int k4 = 0; k4 < RPT / 4; ++k4) {
                        const float4 y4 =
                            *reinterpret_cast<const float4 *>(&ys[buf][(i8 + i) * W + row_of(4 * k4)]);
                        const float4 x4 = kState ? y4 : *reinterpret_cast<const float4 *>(
                                                            &xs[buf][(i8 + i) * W + row_of(4 * k4)]);
                        const float2 yv[2] = {make_float2(y4.x, y4.y), make_float2(y4.z, y4.w)};
                        const float2 xv[2] = {make_float2(x4.x, x4.y), make_float2(x4.z, x4.w)};
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int c = 0; c < NC; ++c) {
                                float2 &sk = s[c][2 * k4 + e];
                                const float2 zz = make_float2(zt[c], zt[c]);
                                sk = is_slow ? tc::fma2(yv[e], zz, sk) : tc::fma2(ff, sk, tc::mul2(yv[e], zz));
                                if (!kState) part[c] = tc::fma2(xv[e], sk, part[c]);
                            }
                    }
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[i * NC + c] = part[c].x + part[c].y;
                }
                // sums over the 8 row groups, of 8 values at once: each step halves the values a lane
                // holds, and lane rg is left with value rg
                if constexpr (!kState) {
#pragma unroll
                    for (int n = 4; n > 0; n >>= 1)
#pragma unroll
                        for (int i = 0; i < n; ++i) {
                            const bool up = rg & n;
                            const float keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
                            acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, n);
                        }
                    os[i8 + rg / NC][col + rg % NC] = acc[0];
                }
            }
        };
        if (slow) walk(std::true_type{});
        else walk(std::false_type{});
        if (kState) continue;       // (the next tile goes to the other buffer)
        __syncthreads();
        for (int e = threadIdx.x; e < nt * kCols; e += kThreads) {
            const int i = e / kCols, c = e % kCols;
            if (z0 + c >= m.Dz) continue;
            const int64_t t = rev ? p.T - 1 - (i0 + i) : i0 + i;
            const int64_t at = ((b * p.T + t) * p.H + h) * m.Dz + z0 + c;
            const float v = of[i + TB - nt] * os[i][c];
            if (m.out_f32) static_cast<float *>(m.out)[at] = v;
            else put(static_cast<T *>(m.out) + at, v);
        }
    }
    if (kState) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) E[seg * e_seg + k * kThreads] = s[k / (RPT / 2)][k % (RPT / 2)];
        return;
    }
    if (!m.fin || seg != sg.n - 1) return;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int k = 0; k < RPT; ++k) {
            const int r = row_of(k), z = z0 + col + c;
            float v = k & 1 ? s[c][k / 2].y : s[c][k / 2].x;
            if (rev) v *= lam;
            if (z < m.Dz && r < m.Dx)
                m.fin[bh * m.Dx * m.Dz + (m.fin_t ? (int64_t)z * m.Dx + r : (int64_t)r * m.Dz + z)] = v;
        }
}

// E(j) -> S(j + 1), in place: a thread takes one pair of values through all segments.
constexpr int kScanBatch = 8;
__global__ void __launch_bounds__(kThreads)
hda_exact_scan_kernel(const float *__restrict__ decay, int64_t H, const Segs sg, int64_t per_seg, int64_t pairs) {
    tc::pdl_launch_dependents();
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= pairs) return;
    const int64_t mbh = e / per_seg;        // map and head
    // (not below the least positive float unless l is zero: an infinite state stays infinite)
    const float g = decay[mbh % H], f = fmaxf(decay_pow(g, (float)sg.len), expf(g) > 0.f ? 0x1p-149f : 0.f);
    float2 *E = sg.E + mbh * (sg.n - 1) * per_seg + e % per_seg;
    tc::pdl_wait_prerequisites();
    float2 s = make_float2(0.f, 0.f);
    for (int j0 = 0; j0 < sg.n - 1; j0 += kScanBatch) {
        float2 v[kScanBatch];
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j)
            if (j0 + j < sg.n - 1) v[j] = E[(j0 + j) * per_seg];
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j) {
            if (j0 + j >= sg.n - 1) break;
            s = j0 + j == 0 ? v[j] : tc::fma2(make_float2(f, f), s, v[j]);
            E[(j0 + j) * per_seg] = s;
        }
    }
}

// Gradients of shared heads: the state heads' parts are added in fp32 in the order of the
// heads, and rounded once. (67 MB of parts: 14 us from cold caches, 4.8 TB/s.)
template <typename T>
__global__ void hda_share_kernel(HdaShare a, HdaShare b, HdaShare c, int64_t BT, int64_t H) {
    tc::pdl_wait_prerequisites();
    const HdaShare s = blockIdx.y == 0 ? a : blockIdx.y == 1 ? b : c;
    const int64_t n = BT * s.heads * (s.D / 4);
    const int rep = (int)(H / s.heads);
    for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n;
         e += (int64_t)gridDim.x * blockDim.x) {
        const int64_t d4 = e % (s.D / 4), th = e / (s.D / 4);   // th = token * heads + head
        const float *ip = s.in + th * rep * s.D + d4 * 4;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r0 = 0; r0 < rep; r0 += 4) {       // (four loads on their way at a time)
            float4 w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r0 + r < rep) w[r] = __ldcs(reinterpret_cast<const float4 *>(ip + (int64_t)(r0 + r) * s.D));
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r0 + r < rep) {
                    v.x += w[r].x;
                    v.y += w[r].y;
                    v.z += w[r].z;
                    v.w += w[r].w;
                }
        }
        put4(static_cast<T *>(s.out) + e * 4, v);
    }
}

constexpr int kTile = 16, kMostSegs = 128;

void exact_dims(const HdaProblem &p, int &dx, int &dz) {
    dx = dz = 0;
    for (int i = 0; i < p.n; ++i) {
        dx = max(dx, p.lin[i].Dx);
        dz = max(dz, p.lin[i].Dz);
    }
}

struct ExactPlan {
    int rows, cols;         // of S in a thread
    Segs g;
};

// Segments of a sequence, and one column of S per thread or kWide (4; with more than 128 rows, 2): one
// is faster for a CTA by itself, four read x and y once for four times the columns. The cost of each
// in ns, set where the choices came out best at 128 rows (one column and four): the token of a lone
// CTA 122 and 270 (measured: 120 and 235); as long as an SM's CTAs are fewer than 1.2 and 1.9, it does
// not depend on them, then it grows in proportion (16 CTAs of one column to an SM: 1330; 4 of four:
// 650); the first kernel's tokens 0.7 of that; 6 us for the two kernels more. (With 120, 235 and 1.45
// CTAs for both, one head of 16384 tokens takes 94 us, not 82, and 8 of 2048 90, not 66.)
ExactPlan exact_plan(const HdaProblem &p, int splits, int sms) {
    int dx, dz;
    exact_dims(p, dx, dz);
    ExactPlan best{};
    best.rows = dx <= 64 ? 8 : dx <= 128 ? 16 : 32;
    double least = 0;
    for (int wide = 0; wide < 2; ++wide) {
        const int cols = wide ? (dx <= 128 ? 4 : 2) : 1, zblocks = (dz + 16 * cols - 1) / (16 * cols);
        const double ctas = (double)(p.B * p.H * p.n) * zblocks, token = wide ? 270 : 122, share = wide ? 1.9 : 1.2;
        int most = (int)min(p.T / (2 * kTile), (int64_t)kMostSegs);
        if (splits > 0) most = min(splits, kMostSegs);
        for (int n = splits > 0 ? most : 1; n <= max(most, 1); ++n) {
            const double walk = token * (double)p.T / n * max(1.0, ctas * n / (share * sms));
            const double cost = n == 1 ? walk : 1.7 * walk + 6000.0;
            if (least > 0 && cost >= least) continue;
            least = cost;
            best.cols = cols;
            best.g.n = n;
            best.g.zblocks = zblocks;
        }
    }
    const int64_t len = (p.T + best.g.n - 1) / best.g.n;
    best.g.len = (len + kTile - 1) / kTile * kTile;
    best.g.n = (int)max((int64_t)1, (p.T + best.g.len - 1) / best.g.len);
    return best;
}
int64_t pairs_per_segment(const ExactPlan &e) { return (int64_t)e.g.zblocks * e.rows * e.cols / 2 * kThreads; }

template <typename T, int RPT, int NC, int TB>
cudaError_t launch_walk(const HdaProblem &p, const Segs &g, cudaStream_t s) {
    // heads of all entries in y, what exceeds its limit in z beside the maps
    const int64_t bh = p.B * p.H, rows = min(bh, (int64_t)65535);
    dim3 grid(g.zblocks * g.n, (unsigned)rows, (unsigned)((bh + rows - 1) / rows * p.n));
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = pdl;
    if (g.n > 1) {
        cfg.gridDim = dim3(g.zblocks * (g.n - 1), grid.y, grid.z);
        cudaError_t e = cudaLaunchKernelEx(&cfg, hda_exact_kernel<T, RPT, NC, TB, true>, p, g);
        if (e != cudaSuccess) return e;
        cfg.numAttrs = 1;
        const int64_t per_seg = (int64_t)g.zblocks * (RPT * NC / 2) * kThreads, pairs = p.n * p.B * p.H * per_seg;
        cfg.gridDim = dim3((unsigned)((pairs + kThreads - 1) / kThreads));
        e = cudaLaunchKernelEx(&cfg, hda_exact_scan_kernel, p.decay, p.H, g, per_seg, pairs);
        if (e != cudaSuccess) return e;
        count_launches(2);
    }
    cfg.gridDim = grid;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, hda_exact_kernel<T, RPT, NC, TB, false>, p, g);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t run_exact(const HdaProblem &p, int splits, int sms, void *ws, cudaStream_t s) {
    ExactPlan plan = exact_plan(p, splits, sms);
    const Segs &g = plan.g;
    plan.g.E = static_cast<float2 *>(ws);
    const bool one = plan.cols == 1;
    if (plan.rows == 8) return one ? launch_walk<T, 8, 1, kTile>(p, g, s) : launch_walk<T, 8, 4, kTile>(p, g, s);
    if (plan.rows == 16) return one ? launch_walk<T, 16, 1, kTile>(p, g, s) : launch_walk<T, 16, 4, kTile>(p, g, s);
    return one ? launch_walk<T, 32, 1, kTile / 2>(p, g, s) : launch_walk<T, 32, 2, kTile / 2>(p, g, s);
}

}  // namespace

size_t hda_exact_workspace_bytes(const HdaProblem &p, int splits, int num_sms) {
    const ExactPlan plan = exact_plan(p, splits, num_sms);
    return (size_t)(plan.g.n - 1) * p.n * p.B * p.H * pairs_per_segment(plan) * sizeof(float2);
}

cudaError_t launch_hda_exact(const HdaProblem &p, int splits, int num_sms, void *ws, cudaStream_t s) {
    return p.io == 0 ? run_exact<__nv_bfloat16>(p, splits, num_sms, ws, s)
                     : run_exact<float>(p, splits, num_sms, ws, s);
}

cudaError_t launch_hda_share(const HdaShare *parts, int n, int64_t BT, int64_t H, int io,
                             cudaStream_t s) {
    if (n == 0 || BT == 0) return cudaSuccess;
    int64_t most = 0;
    for (int i = 0; i < n; ++i) most = max(most, BT * parts[i].heads * (parts[i].D / 4));
    const dim3 grid((unsigned)min((most + 255) / 256, (int64_t)1 << 16), n);
    const HdaShare b = parts[n > 1 ? 1 : 0], c = parts[n > 2 ? 2 : 0];
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    const cudaError_t e =
        io == 0 ? cudaLaunchKernelEx(&cfg, hda_share_kernel<__nv_bfloat16>, parts[0], b, c, BT, H)
                : cudaLaunchKernelEx(&cfg, hda_share_kernel<float>, parts[0], b, c, BT, H);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
