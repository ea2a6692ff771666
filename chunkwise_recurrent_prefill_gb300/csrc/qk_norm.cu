// Norm of queries and keys for each head with the position rotation in the same pass:
//     n = x r w,   r = (s sum x^2 + eps)^-1/2;   pairs (a, b) of n -> (a cos - b sin, b cos + a sin)
// and its gradient, with g the gradient of n (the rotation's transpose of the output's) times w and
// xh = x r:
//     dx = r (g - xh s sum(g xh)),   dw = sum over tokens and heads of (g / w) xh
// Every value is read once and written once, so HBM bandwidth bounds it.
#include <algorithm>

#include "elem.cuh"
#include "gla_internal.h"
#include "launch.h"
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
    tc::pdl_launch_dependents();
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

// ---------------------------------------------------------------- vectors
// Where the rows are on 16 bytes and the rotation's halves are whole vectors: a segment of W lanes (a power of
// two) owns a few heads of a token; a lane has a unit of two vectors of each head, the two that turn together
// (i, i + R / 2), or side by side. The angles of a token are loaded once for its heads, weights once for all
// of a thread's tokens.
struct QkPlan {
    int W;                  // lanes of a segment
    int chunks[2];          // CTAs (grid y) over the heads of q and k
};

// What a lane's unit is.
template <int V>
struct Unit {
    int at[2];              // first elements of its vectors, or -1
    int turn;               // 0: none, 1: halves, 2: pairs
    int angle;              // the first of its angles
    __device__ Unit(const QkProblem &p, int u) {
        const int rot = p.R / (2 * V);          // units of halves
        if (!p.pairs) {
            turn = u < rot;
            angle = u * V;
            at[0] = turn ? u * V : p.R + 2 * (u - rot) * V;
            at[1] = turn ? p.R / 2 + u * V : at[0] + V;
        } else {                                // (R is whole units, or the layout is the plain kernel's)
            at[0] = 2 * u * V;
            at[1] = at[0] + V;
            turn = at[0] < p.R ? 2 : 0;
            angle = u * V;
        }
        for (int i = 0; i < 2; ++i)
            if (at[i] >= p.D) at[i] = -1;
    }
};

// The unit's V angles of a token.
template <int V>
__device__ __forceinline__ void load_angles(const QkProblem &p, int angle, int64_t pos, float (&c)[V], float (&s)[V]) {
    const float4 *cp = reinterpret_cast<const float4 *>(p.cos + pos * (p.R / 2) + angle);
    const float4 *sp = reinterpret_cast<const float4 *>(p.sin + pos * (p.R / 2) + angle);
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 a = __ldg(cp + i / 4), b = __ldg(sp + i / 4);
        c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
        s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
    }
}

// The rotation of a unit (x, y), or with back its transpose.
template <int V, bool kBack>
__device__ __forceinline__ void rotate(int turn, float (&x)[V], float (&y)[V], const float (&c)[V], const float (&s)[V]) {
    if (turn == 1) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float a = x[i], b = y[i], sn = kBack ? -s[i] : s[i];
            x[i] = fmaf(a, c[i], -(b * sn));
            y[i] = fmaf(b, c[i], a * sn);
        }
    } else if (turn == 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float(&v)[V] = i < V / 2 ? x : y;
            const int k = 2 * i % V;
            const float a = v[k], b = v[k + 1], sn = kBack ? -s[i] : s[i];
            v[k] = fmaf(a, c[i], -(b * sn));
            v[k + 1] = fmaf(b, c[i], a * sn);
        }
    }
}

__device__ __forceinline__ float sum_lanes(float v, int W) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < W) v += __shfl_xor_sync(0xffffffffu, v, o);     // (W is the same in the warp)
    return v;
}

// kHeads: heads of a segment at a time.
template <typename T, int V, int kHeads>
__global__ void __launch_bounds__(kThreads)
qk_rows_fwd(const __grid_constant__ QkProblem p, const QkPlan pl, unsigned int *err) {
    using P = Pack<T, V>;
    using R = typename P::raw;
    const int lane = threadIdx.x % pl.W, segs = kThreads / pl.W;
    const int which = (int)blockIdx.y >= pl.chunks[0], h0 = ((int)blockIdx.y - (which ? pl.chunks[0] : 0)) * kHeads;
    const QkHeads &hd = p.t[which];
    const Unit<V> u(p, lane);
    float w[2][V], c[V], sn[V];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) w[k][i] = hd.w && u.at[k] >= 0 ? __ldg(hd.w + u.at[k] + i) : 1.f;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = sn[i] = 0.f;
    const float scale = p.norm == 1 ? 1.f / (float)p.D : 1.f;
    const int64_t tokens = p.B * p.T, step = (int64_t)gridDim.x * segs;
    // (the whole warp walks together: segments past the last token do nothing)
    for (int64_t base = (int64_t)blockIdx.x * segs; base < tokens; base += step) {
        const int64_t token = base + threadIdx.x / pl.W;
        const bool in = token < tokens;
        const int64_t b = in ? token / p.T : 0, t = in ? token - b * p.T : 0;
        int64_t pos = in ? (p.positions ? (int64_t)p.positions[token] : t) : 0;
        const bool known = p.R == 0 || (pos >= 0 && pos < p.P);
        if (!known && in && lane == 0) atomicOr(err, kDevErrPages);
        if (!known) pos = 0;
        const T *x = static_cast<const T *>(hd.x) + b * hd.x_b + t * hd.x_t + (int64_t)h0 * hd.x_h;
        R raw[kHeads][2];
#pragma unroll
        for (int j = 0; j < kHeads; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                raw[j][k] = R{};
                if (in && h0 + j < hd.heads && u.at[k] >= 0)
                    raw[j][k] = *reinterpret_cast<const R *>(x + j * hd.x_h + u.at[k]);
            }
        if (u.turn && p.P > 0) load_angles<V>(p, u.angle, pos, c, sn);
        const int64_t row = token * hd.heads + h0;
        T *out = static_cast<T *>(hd.out) + row * p.D;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if (h0 + j >= hd.heads) break;              // (the same in the CTA)
            float v[2][V];
            P::unpack(raw[j][0], v[0]);
            P::unpack(raw[j][1], v[1]);
            float f = 1.f;
            if (p.norm) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) ss = fmaf(v[0][i], v[0][i], fmaf(v[1][i], v[1][i], ss));
                ss = sum_lanes(ss, pl.W);
                const float m = fmaf(scale, ss, p.eps);
                f = rsqrtf(m);
                // (rare, and decided for the warp: the sum across lanes needs all of them)
                if (__any_sync(0xffffffffu, !(m >= 1e-30f && m <= 1e37f))) {
                    const float e = m < 1.f ? 0x1p100f : 0x1p-100f;
                    float s2 = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float a = v[0][i] * e, d = v[1][i] * e;
                        s2 = fmaf(a, a, fmaf(d, d, s2));
                    }
                    s2 = sum_lanes(s2, pl.W);
                    if (!(m >= 1e-30f && m <= 1e37f)) f = e * rsqrtf(fmaf(scale, s2, p.eps * e * e));
                }
                if (hd.r && in && lane == 0) hd.r[row + j] = known ? f : 0.f;
            }
            if (!in) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) v[k][i] = v[k][i] * f * w[k][i];
            rotate<V, false>(u.turn, v[0], v[1], c, sn);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (u.at[k] < 0) continue;
                *reinterpret_cast<R *>(out + (int64_t)j * p.D + u.at[k]) = known ? P::pack(v[k]) : R{};
            }
        }
    }
}

// Sums of a CTA's tokens go to part[blockIdx.y][blockIdx.x][D].
template <typename T, int V, int kHeads>
__global__ void __launch_bounds__(kThreads)
qk_rows_bwd(const __grid_constant__ QkProblem p, const QkPlan pl, float *part, unsigned int *err) {
    tc::pdl_launch_dependents();
    using P = Pack<T, V>;
    using R = typename P::raw;
    __shared__ float sums[kThreads][V + 1];
    const int lane = threadIdx.x % pl.W, segs = kThreads / pl.W;
    const int which = (int)blockIdx.y >= pl.chunks[0], h0 = ((int)blockIdx.y - (which ? pl.chunks[0] : 0)) * kHeads;
    const QkHeads &hd = p.t[which];
    const Unit<V> u(p, lane);
    float w[2][V], dw[2][V], c[V], sn[V];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = hd.w && u.at[k] >= 0 ? __ldg(hd.w + u.at[k] + i) : 1.f;
            dw[k][i] = 0.f;
        }
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = sn[i] = 0.f;
    const float scale = p.norm == 1 ? 1.f / (float)p.D : 1.f;
    const int64_t tokens = p.B * p.T, step = (int64_t)gridDim.x * segs;
    for (int64_t base = (int64_t)blockIdx.x * segs; base < tokens; base += step) {
        const int64_t token = base + threadIdx.x / pl.W;
        const bool in = token < tokens;
        const int64_t b = in ? token / p.T : 0, t = in ? token - b * p.T : 0;
        int64_t pos = in ? (p.positions ? (int64_t)p.positions[token] : t) : 0;
        const bool known = p.R == 0 || (pos >= 0 && pos < p.P);
        if (!known && in && lane == 0) atomicOr(err, kDevErrPages);
        if (!known) pos = 0;
        const T *x = static_cast<const T *>(hd.x) + b * hd.x_b + t * hd.x_t + (int64_t)h0 * hd.x_h;
        const T *go = static_cast<const T *>(hd.go) + b * hd.g_b + t * hd.g_t + (int64_t)h0 * hd.g_h;
        const int64_t row = token * hd.heads + h0;
        R xr[kHeads][2], gr[kHeads][2];
        float f[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            const bool have = in && h0 + j < hd.heads;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                xr[j][k] = gr[j][k] = R{};
                if (have && u.at[k] >= 0) {
                    if (p.norm) xr[j][k] = *reinterpret_cast<const R *>(x + j * hd.x_h + u.at[k]);
                    gr[j][k] = *reinterpret_cast<const R *>(go + j * hd.g_h + u.at[k]);
                }
            }
            f[j] = have && p.norm ? hd.r[row + j] : 1.f;
        }
        if (u.turn && p.P > 0) load_angles<V>(p, u.angle, pos, c, sn);
        T *out = static_cast<T *>(hd.out) + row * p.D;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if (h0 + j >= hd.heads) break;              // (the same in the CTA)
            float g[2][V], xh[2][V];
            P::unpack(gr[j][0], g[0]);
            P::unpack(gr[j][1], g[1]);
            rotate<V, true>(u.turn, g[0], g[1], c, sn);
            if (p.norm) {
                P::unpack(xr[j][0], xh[0]);
                P::unpack(xr[j][1], xh[1]);
                float dot = 0.f;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        xh[k][i] *= f[j];
                        const float gx = g[k][i] * xh[k][i];
                        if (in && known) dw[k][i] += gx;
                        dot = fmaf(gx, w[k][i], dot);
                    }
                dot = sum_lanes(dot, pl.W) * scale;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) g[k][i] = f[j] * fmaf(-xh[k][i], dot, g[k][i] * w[k][i]);
            }
            if (!in) continue;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (u.at[k] < 0) continue;
                *reinterpret_cast<R *>(out + (int64_t)j * p.D + u.at[k]) = known ? P::pack(g[k]) : R{};
            }
        }
    }
    if (!part) return;
    // the segments of the CTA are added in their order
    float *to = part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) sums[threadIdx.x][i] = dw[k][i];
        __syncthreads();
        for (int e = threadIdx.x; e < pl.W * V; e += kThreads) {
            const Unit<V> o(p, e / V);
            if (o.at[k] < 0) continue;
            float s = 0.f;
            for (int r = 0; r < segs; ++r) s += sums[r * pl.W + e / V][e % V];
            to[o.at[k] + e % V] = s;
        }
    }
}

// dwq and dwk from parts, each added in a fixed order: 32 rows of threads take every 32nd part, then are added.
struct QkSums {
    const float *part[2];
    int64_t n[2], stride[2];
};
__global__ void __launch_bounds__(1024)
qk_sums_kernel(const __grid_constant__ QkProblem p, const __grid_constant__ QkSums q) {
    __shared__ float rows[32][33];
    const int which = blockIdx.y, col = threadIdx.x % 32, row = threadIdx.x / 32, i = blockIdx.x * 32 + col;
    float s = 0.f;
    tc::pdl_wait_prerequisites();
    if (i < p.D) {
        const float *at = q.part[which] + i;
#pragma unroll 8
        for (int64_t k = row; k < q.n[which]; k += 32) s += at[k * q.stride[which]];
    }
    rows[row][col] = s;
    __syncthreads();
    // a warp adds the rows of one column
    s = rows[col][row];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int c = blockIdx.x * 32 + row;
    if (col == 0 && c < p.D && p.t[which].dw) p.t[which].dw[c] = s;
}

int64_t rows_of(const QkProblem &p) { return p.B * p.T * (p.t[0].heads + p.t[1].heads); }

int bwd_parts(const QkProblem &p, int num_sms) {
    return (int)std::min<int64_t>((rows_of(p) + kWarps - 1) / kWarps, 4 * num_sms);
}

bool on16(const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; }

// Whether the vector kernels take the problem: rows on 16 bytes, the rotation in whole units, at most 32 of them.
bool vectors(const QkProblem &p) {
    const int V = p.io == 0 ? 8 : 4, es = p.io == 0 ? 2 : 4;
    if (p.D % V != 0 || (p.D + 2 * V - 1) / (2 * V) > 32 || p.R % (2 * V) != 0) return false;
    if (p.R > 0 && (!on16(p.cos) || !on16(p.sin))) return false;
    for (const QkHeads &t : p.t) {
        if (t.heads == 0) continue;
        if (!on16(t.x) || t.x_b * es % 16 || t.x_t * es % 16 || t.x_h * es % 16) return false;
        if (t.go && (!on16(t.go) || t.g_b * es % 16 || t.g_t * es % 16 || t.g_h * es % 16)) return false;
    }
    return true;
}

constexpr int kFwdHeads = 4, kBwdHeads = 2;

QkPlan plan_of(const QkProblem &p, int heads) {
    const int V = p.io == 0 ? 8 : 4, units = (p.D + 2 * V - 1) / (2 * V);
    QkPlan pl;
    pl.W = 1;
    while (pl.W < units) pl.W *= 2;
    for (int i = 0; i < 2; ++i) pl.chunks[i] = (p.t[i].heads + heads - 1) / heads;
    return pl;
}
// CTAs over the tokens: all resident at once (four to an SM), or one for each few tokens.
unsigned token_ctas(const QkProblem &p, const QkPlan &pl, int num_sms) {
    const int64_t segs = kThreads / pl.W, need = (p.B * p.T + segs - 1) / segs;
    const int64_t most = std::max(1, 4 * num_sms / std::max(1, pl.chunks[0] + pl.chunks[1]));
    return (unsigned)std::min(need, most);
}

}  // namespace

cudaError_t launch_qk_fwd(const QkProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    if (vectors(p)) {
        const QkPlan pl = plan_of(p, kFwdHeads);
        const dim3 grid(token_ctas(p, pl, num_sms), (unsigned)(pl.chunks[0] + pl.chunks[1]));
        if (p.io == 0) qk_rows_fwd<__nv_bfloat16, 8, kFwdHeads><<<grid, kThreads, 0, s>>>(p, pl, dev_err);
        else qk_rows_fwd<float, 4, kFwdHeads><<<grid, kThreads, 0, s>>>(p, pl, dev_err);
    } else {
        const unsigned grid = (unsigned)((rows_of(p) + kWarps - 1) / kWarps);
        if (p.io == 0) qk_plain_fwd<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, dev_err);
        else qk_plain_fwd<float><<<grid, kThreads, 0, s>>>(p, dev_err);
    }
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// (what either kernel needs: the one that runs depends on the pointers)
size_t qk_bwd_workspace_bytes(const QkProblem &p, int num_sms) {
    if (!p.norm) return 0;
    const QkPlan pl = plan_of(p, kBwdHeads);
    const size_t plain = (size_t)bwd_parts(p, num_sms) * 2,
                 vec = pl.W > 32 ? 0 : (size_t)token_ctas(p, pl, num_sms) * (pl.chunks[0] + pl.chunks[1]);
    return std::max(plain, vec) * p.D * sizeof(float);
}

template <typename T>
static cudaError_t run_bwd(const QkProblem &p, float *part, int num_sms, unsigned int *err, cudaStream_t s) {
    QkSums sums{};
    if (vectors(p)) {
        const QkPlan pl = plan_of(p, kBwdHeads);
        const dim3 grid(token_ctas(p, pl, num_sms), (unsigned)(pl.chunks[0] + pl.chunks[1]));
        qk_rows_bwd<T, 16 / sizeof(T), kBwdHeads><<<grid, kThreads, 0, s>>>(p, pl, part, err);
        for (int i = 0; i < 2; ++i) {
            sums.part[i] = part + (i ? (size_t)pl.chunks[0] * grid.x * p.D : 0);
            sums.n[i] = (int64_t)pl.chunks[i] * grid.x;
            sums.stride[i] = p.D;
        }
    } else {
        const int parts = bwd_parts(p, num_sms);
        const size_t smem = 2 * kWarps * (size_t)p.D * sizeof(float);
        const cudaError_t e = cudaFuncSetAttribute(qk_plain_bwd<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        qk_plain_bwd<T><<<parts, kThreads, smem, s>>>(p, part, err);
        for (int i = 0; i < 2; ++i) {
            sums.part[i] = part + (i ? p.D : 0);
            sums.n[i] = parts;
            sums.stride[i] = 2 * p.D;
        }
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    return part ? launch(qk_sums_kernel, dim3((p.D + 31) / 32, 2), 1024, 0, true, s, p, sums) : e;
}

cudaError_t launch_qk_bwd(const QkProblem &p, void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    float *part = p.norm && (p.t[0].dw || p.t[1].dw) ? static_cast<float *>(ws) : nullptr;
    return p.io == 0 ? run_bwd<__nv_bfloat16>(p, part, num_sms, dev_err, s)
                     : run_bwd<float>(p, part, num_sms, dev_err, s);
}

}  // namespace gla
