// Selective state space scan: N states per channel, whose decays are inputs,
//     h_t = a_t h_{t-1} + d_t u_t B_t,   a_t = e^(d_t A),   y_t = C_t . h_t + D u_t,   o_t = y_t silu(z_t)
// and its gradients. With dy = d_o silu(z), G_t the gradient of h_t and G'_t = a_t G_t what it passes
// to the token before:
//     G_t = C_t dy_t + G'_{t+1},   w_t = G'_t h_{t-1}
//     dd_t = sum_n w_t A + u_t sum_n G_t B_t,   du_t = d_t sum_n G_t B_t + D dy_t
//     dA = sum_t w_t d_t,   dB_t = sum_c G_t d_t u_t,   dC_t = sum_c h_t dy_t
//
// A ring of warps: a CTA owns 32 channels (one per lane) of a sequence, and its warps take chunks of
// kTok tokens in turn. All that a chunk can do without the state (loads, step sizes, the exponentials
// and inputs of four states at a time) runs while the chunks before it are still at work; the
// four states then come from the warp before through shared memory, walk over the chunk's tokens in
// registers and go on to the next warp. So a sequence is walked once, and each exponential is computed
// once, although all warps work at the same time. Backwards the ring turns the other way.
#include <cuda_bf16.h>

#include <algorithm>

#include "elem.cuh"
#include "gla_internal.h"
#include "ssm.h"

namespace gla {
namespace {

constexpr int kTok = 8;             // tokens of a chunk
constexpr int kLanes = 32;          // channels of a CTA
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

using tc::fma2;
using tc::mul2;
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Quad {                       // four states of a channel
    float2 a, b;
};
__device__ __forceinline__ Quad quad(float4 v) { return Quad{make_float2(v.x, v.y), make_float2(v.z, v.w)}; }
__device__ __forceinline__ float4 vec4(const Quad &q) { return make_float4(q.a.x, q.a.y, q.b.x, q.b.y); }
__device__ __forceinline__ Quad operator*(const Quad &x, const Quad &y) { return Quad{mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ Quad operator*(const Quad &x, float y) { return Quad{mul2(x.a, both(y)), mul2(x.b, both(y))}; }
__device__ __forceinline__ Quad fmaq(const Quad &x, const Quad &y, const Quad &z) {
    return Quad{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)};
}
__device__ __forceinline__ Quad fmaq(const Quad &x, float y, const Quad &z) {
    return Quad{fma2(x.a, both(y), z.a), fma2(x.b, both(y), z.b)};
}
__device__ __forceinline__ Quad exp2q(const Quad &x) {
    return Quad{make_float2(ex2(x.a.x), ex2(x.a.y)), make_float2(ex2(x.b.x), ex2(x.b.y))};
}
// x . y added to a pair of sums
__device__ __forceinline__ float2 dotq(const Quad &x, const Quad &y, float2 s) { return fma2(x.b, y.b, fma2(x.a, y.a, s)); }

// Four consecutive values of a row of N from value n0 on (zero past the end).
__device__ __forceinline__ float4 load_quad(const float *row, int n0, int N) {
    if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0)
        return *reinterpret_cast<const float4 *>(row + n0);
    return make_float4(n0 < N ? row[n0] : 0.f, n0 + 1 < N ? row[n0 + 1] : 0.f, n0 + 2 < N ? row[n0 + 2] : 0.f,
                       n0 + 3 < N ? row[n0 + 3] : 0.f);
}
__device__ __forceinline__ void store_quad(float *row, int n0, int N, float4 v) {
    if (N % 4 == 0) {
        *reinterpret_cast<float4 *>(row + n0) = v;
        return;
    }
    if (n0 < N) row[n0] = v.x;
    if (n0 + 1 < N) row[n0 + 1] = v.y;
    if (n0 + 2 < N) row[n0 + 2] = v.z;
    if (n0 + 3 < N) row[n0 + 3] = v.w;
}

// A times log2 e, with infinities brought to the largest float: a step of zero then keeps the state.
__device__ __forceinline__ float scale_a(float a) { return fminf(fmaxf(a * kLog2e, -3.4028235e38f), 3.4028235e38f); }

__device__ __forceinline__ float step_size(float x, int softplus) {
    return softplus ? fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))) : x;
}

// Which sequence, group and channels a CTA has.
struct Tiles {
    int per_group;                  // CTAs of 32 channels for a group
    int64_t all;                    // of a sequence
};
__host__ __device__ inline Tiles tiles_of(int64_t C, int64_t G) {
    const int64_t cg = C / G;
    const int64_t n = (cg + kLanes - 1) / kLanes;
    return Tiles{(int)n, n * G};
}

// Shared memory of a ring of W warps with Q quads of states:
//   slot[W][Q][32] float4: what a warp hands on;  A[Q][32] float4;  rows[W][2][kTok][4 Q]: B and C of
//   a warp's chunk;  sums[W][Q][32] float4 (backward: dA);  bar[W][Q]
struct Ring {
    float4 *slot, *A, *sums;
    float *rows;
    uint64_t *bar;
    static __host__ __device__ size_t bytes(int W, int Q, bool backward) {
        return (size_t)W * Q * kLanes * 16 * (backward ? 2 : 1) + (size_t)Q * kLanes * 16 +
               (size_t)W * 2 * kTok * 4 * Q * 4 + (size_t)W * Q * 8;
    }
    __device__ Ring(unsigned char *smem, int W, int Q, bool backward) {
        slot = reinterpret_cast<float4 *>(smem);
        A = slot + W * Q * kLanes;
        sums = A + Q * kLanes;
        rows = reinterpret_cast<float *>(sums + (backward ? W * Q * kLanes : 0));
        bar = reinterpret_cast<uint64_t *>(rows + W * 2 * kTok * 4 * Q);
    }
};

// B and C of the chunk's tokens as floats: to[2][kTok][4 Q], zero past the last token and state.
template <typename T>
__device__ __forceinline__ void load_rows(const SsmProblem &p, int64_t b, int64_t g, int64_t t0, int Q, float *to) {
    const int lane = threadIdx.x % 32, NP = 4 * Q;
    for (int k = lane; k < kTok * NP; k += 32) {
        const int i = k / NP, n = k - i * NP;
        const bool in = t0 + i < p.T && n < p.N;
        const int64_t at = g * p.N + n;
        to[k] = in ? get(static_cast<const T *>(p.Bm.p) + b * p.Bm.b + (t0 + i) * p.Bm.t + at) : 0.f;
        to[kTok * NP + k] = in ? get(static_cast<const T *>(p.Cm.p) + b * p.Cm.b + (t0 + i) * p.Cm.t + at) : 0.f;
    }
}

// kOut: outputs and the last state; else the states before each chunk go to marks
// [B][chunks][tiles][Q][32] float4.
template <typename T, int kQ, bool kOut>
__global__ void __launch_bounds__(256)
ssm_fwd_kernel(const __grid_constant__ SsmProblem p, float4 *marks, unsigned int *err) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int W = blockDim.x / 32, Q = kQ ? kQ : (p.N + 3) / 4, NP = 4 * Q;
    const Ring ring(smem, W, Q, false);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G);
    const int64_t b = blockIdx.x / tl.all, tile = blockIdx.x % tl.all, g = tile / tl.per_group;
    const int64_t cg = p.C / p.G, in_group = (tile % tl.per_group) * kLanes + lane;
    const bool live = in_group < cg;
    const int64_t c = g * cg + (live ? in_group : 0);
    for (int q = w; q < Q; q += W) {
        const float4 a = load_quad(p.A + c * p.N, 4 * q, p.N);
        ring.A[q * kLanes + lane] = make_float4(scale_a(a.x), scale_a(a.y), scale_a(a.z), scale_a(a.w));
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < W * Q; ++i) tc::mbar_init(ring.bar + i, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
    float *rows = ring.rows + w * 2 * kTok * NP;
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    const int64_t state = (b * p.C + c) * p.N;
    const int prev = w == 0 ? W - 1 : w - 1;
    bool dead = false;
    for (int64_t ch = w; ch < chunks; ch += W) {
        const int64_t t0 = ch * kTok;
        float u[kTok], d[kTok], du[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const bool in = live && t0 + i < p.T;
            u[i] = in ? get(static_cast<const T *>(p.u.p) + b * p.u.b + (t0 + i) * p.u.t + c) : 0.f;
            d[i] = in ? step_size(get(static_cast<const T *>(p.dt.p) + b * p.dt.b + (t0 + i) * p.dt.t + c) + bias,
                                  p.softplus)
                      : 0.f;
            du[i] = d[i] * u[i];
        }
        __syncwarp();
        load_rows<T>(p, b, g, t0, Q, rows);
        __syncwarp();
        float2 y[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) y[i] = both(0.f);
        const uint32_t parity = (uint32_t)((ch - 1) / W) & 1u;
        for (int q = 0; q < Q; ++q) {
            const Quad A = quad(ring.A[q * kLanes + lane]);
            Quad a[kTok], x[kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                a[i] = exp2q(A * d[i]);
                x[i] = quad(*reinterpret_cast<const float4 *>(rows + i * NP + 4 * q)) * du[i];
            }
            Quad h;
            if (ch == 0) {
                h = quad(p.h0 && live ? load_quad(p.h0 + state, 4 * q, p.N) : make_float4(0.f, 0.f, 0.f, 0.f));
            } else {
                if (!dead && !tc::mbar_wait(ring.bar + prev * Q + q, parity)) {
                    dead = true;
                    atomicOr(err, kDevErrTimeout);
                }
                h = quad(ring.slot[(prev * Q + q) * kLanes + lane]);
            }
            if (!kOut) marks[(((b * chunks + ch) * tl.all + tile) * Q + q) * kLanes + lane] = vec4(h);
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                h = fmaq(a[i], h, x[i]);
                x[i] = h;
            }
            if (ch + 1 < chunks) {
                ring.slot[(w * Q + q) * kLanes + lane] = vec4(h);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(ring.bar + w * Q + q);
            } else if (kOut && p.hT && live) {
                store_quad(p.hT + state, 4 * q, p.N, vec4(h));
            }
            if (kOut) {
#pragma unroll
                for (int i = 0; i < kTok; ++i)
                    y[i] = dotq(x[i], quad(*reinterpret_cast<const float4 *>(rows + (kTok + i) * NP + 4 * q)), y[i]);
            }
        }
        if (kOut) {
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                if (!live || t0 + i >= p.T) break;
                float o = y[i].x + y[i].y;
                if (p.D) o = fmaf(D, u[i], o);
                if (p.z.p) {
                    const float z = get(static_cast<const T *>(p.z.p) + b * p.z.b + (t0 + i) * p.z.t + c);
                    o *= z * logistic<T>(z);
                }
                put(static_cast<T *>(p.o) + (b * p.T + t0 + i) * p.C + c, o);
            }
        }
    }
}

// Sums over the warp's lanes of 32 values each: lane i gets that of value i.
__device__ __forceinline__ float sum_values(float (&v)[32]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float send = up ? v[i] : v[i + s], keep = up ? v[i + s] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    return v[0];
}

// Where the backward kernel leaves what is summed later, all float:
//   rows [tiles][B T][2][4 Q]: dB and dC of a tile's channels
//   chan [B][C][N + 2]: dA, then dD and ddt_bias
struct Parts {
    float *rows, *chan;
};

template <typename T, int kQ>
__global__ void __launch_bounds__(256)
ssm_bwd_kernel(const __grid_constant__ SsmProblem p, const float4 *marks, const Parts parts, unsigned int *err) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float2 chan[8][kLanes];
    const int W = blockDim.x / 32, Q = kQ ? kQ : (p.N + 3) / 4, NP = 4 * Q;
    const Ring ring(smem, W, Q, true);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G);
    const int64_t b = blockIdx.x / tl.all, tile = blockIdx.x % tl.all, g = tile / tl.per_group;
    const int64_t cg = p.C / p.G, in_group = (tile % tl.per_group) * kLanes + lane;
    const bool live = in_group < cg;
    const int64_t c = g * cg + (live ? in_group : 0);
    for (int q = w; q < Q; q += W) {
        const float4 a = load_quad(p.A + c * p.N, 4 * q, p.N);
        ring.A[q * kLanes + lane] = make_float4(scale_a(a.x), scale_a(a.y), scale_a(a.z), scale_a(a.w));
    }
    for (int q = 0; q < Q; ++q) ring.sums[(w * Q + q) * kLanes + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (threadIdx.x == 0) {
        for (int i = 0; i < W * Q; ++i) tc::mbar_init(ring.bar + i, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;
    float *rows = ring.rows + w * 2 * kTok * NP;
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    const int64_t state = (b * p.C + c) * p.N;
    const int prev = w == 0 ? W - 1 : w - 1;
    float dD = 0.f, dbias = 0.f;
    bool dead = false;
    for (int64_t step = w; step < chunks; step += W) {
        const int64_t ch = chunks - 1 - step, t0 = ch * kTok;
        float u[kTok], raw[kTok], d[kTok], go[kTok], dy[kTok], z[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const bool in = live && t0 + i < p.T;
            const int64_t t = t0 + i;
            u[i] = in ? get(static_cast<const T *>(p.u.p) + b * p.u.b + t * p.u.t + c) : 0.f;
            raw[i] = in ? get(static_cast<const T *>(p.dt.p) + b * p.dt.b + t * p.dt.t + c) + bias : 0.f;
            d[i] = in ? step_size(raw[i], p.softplus) : 0.f;
            go[i] = in ? get(static_cast<const T *>(p.go.p) + b * p.go.b + t * p.go.t + c) : 0.f;
            z[i] = in && p.z.p ? get(static_cast<const T *>(p.z.p) + b * p.z.b + t * p.z.t + c) : 0.f;
            dy[i] = p.z.p ? go[i] * z[i] * logistic<T>(z[i]) : go[i];
        }
        __syncwarp();
        load_rows<T>(p, b, g, t0, Q, rows);
        __syncwarp();
        float2 y[kTok], gB[kTok], wA[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) y[i] = gB[i] = wA[i] = both(0.f);
        const uint32_t parity = (uint32_t)((step - 1) / W) & 1u;
        // rows of this tile's dB and dC: lane i sums value i % 4 of token i / 4
        float *out = parts.rows + ((tile * p.B + b) * p.T + t0 + lane / 4) * 2 * NP + lane % 4;
        const bool row_in = t0 + lane / 4 < p.T;
        for (int q = 0; q < Q; ++q) {
            const Quad A = quad(ring.A[q * kLanes + lane]);
            Quad h = quad(marks[(((b * chunks + ch) * tl.all + tile) * Q + q) * kLanes + lane]);
            Quad a[kTok], before[kTok];
            float v[4 * kTok];
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const Quad Bv = quad(*reinterpret_cast<const float4 *>(rows + i * NP + 4 * q));
                const Quad Cv = quad(*reinterpret_cast<const float4 *>(rows + (kTok + i) * NP + 4 * q));
                a[i] = exp2q(A * d[i]);
                before[i] = h;
                h = fmaq(a[i], h, Bv * (d[i] * u[i]));
                y[i] = dotq(h, Cv, y[i]);
                const Quad e = h * dy[i];
                v[4 * i] = e.a.x;
                v[4 * i + 1] = e.a.y;
                v[4 * i + 2] = e.b.x;
                v[4 * i + 3] = e.b.y;
            }
            const float dC = sum_values(v);
            Quad G;
            if (step == 0) {
                G = quad(p.dhT && live ? load_quad(p.dhT + state, 4 * q, p.N) : make_float4(0.f, 0.f, 0.f, 0.f));
            } else {
                if (!dead && !tc::mbar_wait(ring.bar + prev * Q + q, parity)) {
                    dead = true;
                    atomicOr(err, kDevErrTimeout);
                }
                G = quad(ring.slot[(prev * Q + q) * kLanes + lane]);
            }
            Quad dA = quad(ring.sums[(w * Q + q) * kLanes + lane]);
#pragma unroll
            for (int i = kTok - 1; i >= 0; --i) {
                const Quad Bv = quad(*reinterpret_cast<const float4 *>(rows + i * NP + 4 * q));
                const Quad Cv = quad(*reinterpret_cast<const float4 *>(rows + (kTok + i) * NP + 4 * q));
                G = fmaq(Cv, dy[i], G);
                gB[i] = dotq(G, Bv, gB[i]);
                const Quad e = G * (d[i] * u[i]);
                v[4 * i] = e.a.x;
                v[4 * i + 1] = e.a.y;
                v[4 * i + 2] = e.b.x;
                v[4 * i + 3] = e.b.y;
                G = a[i] * G;
                const Quad wt = G * before[i];
                wA[i] = dotq(wt, A, wA[i]);
                dA = fmaq(wt, d[i], dA);
            }
            ring.sums[(w * Q + q) * kLanes + lane] = vec4(dA);
            if (ch > 0) {
                ring.slot[(w * Q + q) * kLanes + lane] = vec4(G);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(ring.bar + w * Q + q);
            } else if (p.dh0 && live) {
                store_quad(p.dh0 + state, 4 * q, p.N, vec4(G));
            }
            const float dB = sum_values(v);
            if (row_in) {
                out[4 * q] = dB;
                out[NP + 4 * q] = dC;
            }
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (!live || t0 + i >= p.T) break;
            const int64_t at = (b * p.T + t0 + i) * p.C + c;
            const float gb = gB[i].x + gB[i].y;
            float ddt = fmaf(wA[i].x + wA[i].y, kLn2, u[i] * gb), du = d[i] * gb;
            if (p.softplus) ddt *= logistic<float>(raw[i]);
            if (p.D) du = fmaf(D, dy[i], du);
            put(static_cast<T *>(p.du) + at, du);
            put(static_cast<T *>(p.ddt) + at, ddt);
            dbias += ddt;
            dD = fmaf(dy[i], u[i], dD);
            if (p.dz) {
                float yy = y[i].x + y[i].y;
                if (p.D) yy = fmaf(D, u[i], yy);
                put(static_cast<T *>(p.dz) + at, go[i] * yy * act_grad<T>(z[i], 1));
            }
        }
    }
    chan[w][lane] = make_float2(dD, dbias);
    __syncthreads();
    if (!live) return;
    float *to = parts.chan + (b * p.C + c) * (p.N + 2);
    for (int n = w; n < p.N; n += W) {
        float s = 0.f;
        for (int i = 0; i < W; ++i)
            s += reinterpret_cast<const float *>(ring.sums + (i * Q + n / 4) * kLanes + lane)[n % 4];
        to[n] = s;
    }
    if (w == 0) {
        for (int i = 1; i < W; ++i) {
            dD += chan[i][lane].x;
            dbias += chan[i][lane].y;
        }
        to[p.N] = dD;
        to[p.N + 1] = dbias;
    }
}

// dB and dC from the tiles' parts, each added in order.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_rows_kernel(const __grid_constant__ SsmProblem p, const Parts parts) {
    const int NP = (p.N + 3) / 4 * 4;
    const Tiles tl = tiles_of(p.C, p.G);
    const int64_t rows = p.B * p.T, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = id % NP, k = id / NP % 2, g = id / (2 * NP) % p.G, row = id / (2 * NP) / p.G;
    if (row >= rows || n >= p.N) return;
    float s = 0.f;
    for (int i = 0; i < tl.per_group; ++i)
        s += parts.rows[(((g * tl.per_group + i) * rows + row) * 2 + k) * NP + n];
    put(static_cast<T *>(k ? p.dCm : p.dBm) + (row * p.G + g) * p.N + n, s);
}
// dA, dD and ddt_bias from the batch entries' parts.
__global__ void __launch_bounds__(256)
ssm_chan_kernel(const __grid_constant__ SsmProblem p, const Parts parts) {
    const int64_t w = p.N + 2, id = (int64_t)blockIdx.x * 256 + threadIdx.x, c = id / w, n = id % w;
    if (c >= p.C) return;
    float s = 0.f;
    for (int64_t b = 0; b < p.B; ++b) s += parts.chan[(b * p.C + c) * w + n];
    if (n < p.N) p.dA[c * p.N + n] = s;
    else if (n == p.N) { if (p.dD) p.dD[c] = s; }
    else if (p.dbias) p.dbias[c] = s;
}

// One token of each row on the pages of a pool. kL lanes (a power of two) own a channel, four states
// each (more where N > 4 kL); their outputs are added by shuffles.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_step_kernel(const __grid_constant__ SsmProblem p, int lanes, unsigned int *err) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int l = (int)(id % lanes);
    const int64_t c = id / lanes % p.C, r = id / lanes / p.C;
    const bool in = r < p.B;
    const int64_t slot = !in ? -1 : p.slots ? p.slots[r] : r;
    const bool live = slot >= 0 && slot < p.P;
    if (in && slot >= p.P && c == 0 && l == 0) atomicOr(err, kDevErrPages);
    float y = 0.f, u = 0.f;
    if (live) {
        const int64_t g = c / (p.C / p.G);
        u = get(static_cast<const T *>(p.u.p) + r * p.u.b + c);
        const float d = step_size(get(static_cast<const T *>(p.dt.p) + r * p.dt.b + c) + (p.dt_bias ? p.dt_bias[c] : 0.f),
                                  p.softplus);
        float *S = p.S + (slot * p.C + c) * p.N;
        const T *Bp = static_cast<const T *>(p.Bm.p) + r * p.Bm.b + g * p.N;
        const T *Cp = static_cast<const T *>(p.Cm.p) + r * p.Cm.b + g * p.N;
        float2 s = both(0.f);
        for (int n0 = 4 * l; n0 < p.N; n0 += 4 * lanes) {
            const float4 a = load_quad(p.A + c * p.N, n0, p.N);
            const Quad A{make_float2(scale_a(a.x), scale_a(a.y)), make_float2(scale_a(a.z), scale_a(a.w))};
            float Bv[4], Cv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                Bv[j] = n0 + j < p.N ? get(Bp + n0 + j) : 0.f;
                Cv[j] = n0 + j < p.N ? get(Cp + n0 + j) : 0.f;
            }
            const Quad x = Quad{make_float2(Bv[0], Bv[1]), make_float2(Bv[2], Bv[3])} * (d * u);
            const Quad h = fmaq(exp2q(A * d), quad(load_quad(S, n0, p.N)), x);
            store_quad(S, n0, p.N, vec4(h));
            s = dotq(h, Quad{make_float2(Cv[0], Cv[1]), make_float2(Cv[2], Cv[3])}, s);
        }
        y = s.x + s.y;
    }
    for (int o = lanes / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!in || l != 0) return;
    if (live) {
        if (p.D) y = fmaf(p.D[c], u, y);
        if (p.z.p) {
            const float z = get(static_cast<const T *>(p.z.p) + r * p.z.b + c);
            y *= z * logistic<T>(z);
        }
    }
    put(static_cast<T *>(p.o) + r * p.C + c, y);
}

int quads(const SsmProblem &p) { return (p.N + 3) / 4; }

// Warps of a ring: at most one for each chunk, and what shared memory holds.
int ring_warps(const SsmProblem &p) {
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    return (int)std::min<int64_t>(quads(p) > 16 ? 4 : 8, chunks);
}

struct BwdWorkspace {
    size_t marks, rows, chan, all;
};
BwdWorkspace bwd_workspace(const SsmProblem &p) {
    auto round = [](size_t n) { return (n + 255) & ~size_t(255); };
    const Tiles tl = tiles_of(p.C, p.G);
    const size_t chunks = (size_t)((p.T + kTok - 1) / kTok), Q = (size_t)quads(p);
    BwdWorkspace w;
    w.marks = round((size_t)p.B * chunks * tl.all * Q * kLanes * 16);
    w.rows = round((size_t)tl.all * p.B * p.T * 2 * 4 * Q * 4);
    w.chan = round((size_t)p.B * p.C * (p.N + 2) * 4);
    w.all = w.marks + w.rows + w.chan;
    return w;
}

template <typename T, int kQ, bool kOut>
cudaError_t run_fwd(const SsmProblem &p, float4 *marks, unsigned int *err, cudaStream_t s) {
    const int W = ring_warps(p);
    const size_t smem = Ring::bytes(W, quads(p), false);
    const cudaError_t e = cudaFuncSetAttribute(ssm_fwd_kernel<T, kQ, kOut>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ssm_fwd_kernel<T, kQ, kOut><<<(unsigned)(p.B * tiles_of(p.C, p.G).all), 32 * W, smem, s>>>(p, marks, err);
    return cudaGetLastError();
}
template <bool kOut>
cudaError_t fwd(const SsmProblem &p, float4 *marks, unsigned int *err, cudaStream_t s) {
    cudaError_t e;
    if (p.io == 0)
        e = quads(p) == 4 ? run_fwd<__nv_bfloat16, 4, kOut>(p, marks, err, s)
                          : run_fwd<__nv_bfloat16, 0, kOut>(p, marks, err, s);
    else
        e = quads(p) == 4 ? run_fwd<float, 4, kOut>(p, marks, err, s) : run_fwd<float, 0, kOut>(p, marks, err, s);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T, int kQ>
cudaError_t run_bwd(const SsmProblem &p, const float4 *marks, const Parts &parts, unsigned int *err, cudaStream_t s) {
    const int W = ring_warps(p);
    const size_t smem = Ring::bytes(W, quads(p), true);
    cudaError_t e = cudaFuncSetAttribute(ssm_bwd_kernel<T, kQ>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    const Tiles tl = tiles_of(p.C, p.G);
    ssm_bwd_kernel<T, kQ><<<(unsigned)(p.B * tl.all), 32 * W, smem, s>>>(p, marks, parts, err);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t rows = p.B * p.T * p.G * 2 * 4 * quads(p), chan = p.C * (p.N + 2);
    ssm_rows_kernel<T><<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(p, parts);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_chan_kernel<<<(unsigned)((chan + 255) / 256), 256, 0, s>>>(p, parts);
    return cudaGetLastError();
}

}  // namespace

size_t ssm_fwd_workspace_bytes(const SsmProblem &, int, int) { return 0; }
size_t ssm_bwd_workspace_bytes(const SsmProblem &p, int, int) { return bwd_workspace(p).all; }

cudaError_t launch_ssm_fwd(const SsmProblem &p, int, int, void *, unsigned int *dev_err, cudaStream_t s) {
    return fwd<true>(p, nullptr, dev_err, s);
}

cudaError_t launch_ssm_bwd(const SsmProblem &p, int, int, void *ws, unsigned int *dev_err, cudaStream_t s) {
    const BwdWorkspace lay = bwd_workspace(p);
    char *at = static_cast<char *>(ws);
    float4 *marks = reinterpret_cast<float4 *>(at);
    const Parts parts{reinterpret_cast<float *>(at + lay.marks), reinterpret_cast<float *>(at + lay.marks + lay.rows)};
    cudaError_t e = fwd<false>(p, marks, dev_err, s);
    if (e != cudaSuccess) return e;
    if (p.io == 0)
        e = quads(p) == 4 ? run_bwd<__nv_bfloat16, 4>(p, marks, parts, dev_err, s)
                          : run_bwd<__nv_bfloat16, 0>(p, marks, parts, dev_err, s);
    else
        e = quads(p) == 4 ? run_bwd<float, 4>(p, marks, parts, dev_err, s)
                          : run_bwd<float, 0>(p, marks, parts, dev_err, s);
    if (e == cudaSuccess) count_launches(3);
    return e;
}

cudaError_t launch_ssm_step(const SsmProblem &p, int, unsigned int *dev_err, cudaStream_t s) {
    int lanes = 1;
    while (lanes < 32 && 4 * lanes < p.N) lanes *= 2;
    const int64_t n = p.B * p.C * lanes;
    const unsigned grid = (unsigned)((n + 255) / 256);
    if (p.io == 0) ssm_step_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p, lanes, dev_err);
    else ssm_step_kernel<float><<<grid, 256, 0, s>>>(p, lanes, dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
