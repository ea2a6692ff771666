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
#include "tma_host.h"

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
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
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
    tc::pdl_wait_prerequisites();
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
// Where the rows are on 16 bytes and the rotation's halves are whole vectors: W lanes (a power of two) own a head, a
// lane a unit of two of its vectors, the two that turn together (i, i + R / 2), or side by side. An item of a warp is
// kHeads heads of 32 / W tokens (at most 4 KB), which TMA brings while the items before it are worked on: what is on its
// way does not cost registers. The heads of a token share its angles, in registers; a CTA keeps to the same heads, so
// that weights are loaded once.
// Measured: 16384 tokens of 16 + 4 heads of 128, bf16 (177 MB): 34.6 us, 5.1 TB/s (fp32 58 us, 5.9); gradients of 8 x 1023 tokens of 16 + 16
// heads of 64 (102 MB): 22.4 us with the sums. Items in registers instead, without packed arithmetic: 37.8 and 27.4.
// Heads of an item: 2 forward 40.4, 8 50.2; backward 1 26.9, 4 29.6. Three items ahead 35.5, three CTAs to an SM
// 37.2; all heads of a token to warps side by side 35.2 and 26.8 (more addresses, and sums of both weights in each CTA).
constexpr int kFwdHeads = 4, kBwdHeads = 2, kAhead = 2;

struct QkPlan {
    int W;                  // lanes of a head
    int chunks[2];          // groups of heads (grid y): of q, of k
    int tiles;              // items of a batch entry
    int box, box_heads;     // values and heads of a TMA load
};
struct QkMaps {
    CUtensorMap x[2], go[2];        // [B, T, heads, D]
};

// What a lane's unit is.
template <int V, bool kPairs>
struct Unit {
    int at[2];              // first elements of its vectors, or -1
    bool turn;
    int angle;              // the first of its angles
    __device__ Unit(const QkProblem &p, int u) {
        const int rot = p.R / (2 * V);          // units that turn
        turn = u < rot;
        angle = u * V;
        at[0] = kPairs ? 2 * u * V : turn ? u * V : p.R + 2 * (u - rot) * V;
        at[1] = !kPairs && turn ? p.R / 2 + u * V : at[0] + V;
        for (int i = 0; i < 2; ++i)
            if (at[i] >= p.D) at[i] = -1;
    }
};

// Vectors of V values as pairs for the packed arithmetic.
template <int V>
using Pairs = float2[V / 2];
template <typename T, int V>
__device__ __forceinline__ void unpack(typename Pack<T, V>::raw r, Pairs<V> &v) {
    float f[V];
    Pack<T, V>::unpack(r, f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::raw pack(const Pairs<V> &v) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i % 2 ? v[i / 2].y : v[i / 2].x;
    return Pack<T, V>::pack(f);
}

// The unit's V angles of a token; back: those of the opposite rotation.
template <int V>
struct Angles {
    Pairs<V> c, s, ns;          // (ns: -s)
    __device__ __forceinline__ void load(const QkProblem &p, int angle, int64_t pos, bool back) {
        const float4 *cp = reinterpret_cast<const float4 *>(p.cos + pos * (p.R / 2) + angle);
        const float4 *sp = reinterpret_cast<const float4 *>(p.sin + pos * (p.R / 2) + angle);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 a = __ldg(cp + i), b = __ldg(sp + i);
            c[2 * i] = make_float2(a.x, a.y), c[2 * i + 1] = make_float2(a.z, a.w);
            s[2 * i] = make_float2(b.x, b.y), s[2 * i + 1] = make_float2(b.z, b.w);
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 n = make_float2(-s[i].x, -s[i].y);
            if (back) ns[i] = s[i], s[i] = n;
            else ns[i] = n;
        }
    }
    // of halves: (x, y) -> (x c - y s, y c + x s)
    template <bool kPairs>
    __device__ __forceinline__ void rotate(Pairs<V> &x, Pairs<V> &y) const {
        if (!kPairs) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 a = x[i], b = y[i];
                x[i] = tc::fma2(b, ns[i], tc::mul2(a, c[i]));
                y[i] = tc::fma2(a, s[i], tc::mul2(b, c[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float2 &v = i < V / 2 ? x[i] : y[i - V / 2];
                const float a = v.x, b = v.y, ci = i % 2 ? c[i / 2].y : c[i / 2].x, si = i % 2 ? s[i / 2].y : s[i / 2].x;
                v = make_float2(fmaf(b, -si, a * ci), fmaf(a, si, b * ci));
            }
        }
    }
};


__device__ __forceinline__ float sum_lanes(float v, int W) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < W) v += __shfl_xor_sync(0xffffffffu, v, o);     // (W is the same in the warp)
    return v;
}

// A warp's items, kAhead of them on their way: kTensors tensors [32 / W][kHeads][D] each.
template <typename T, int kTensors, int kHeads>
struct Items {
    T *stage;
    uint64_t *full;
    int bytes;              // of a tensor of an item
    int step, step_b, step_tile;
    int64_t all;
    struct Place {
        int64_t at;         // b tiles + tile
        int b, tile;
    } now, next;
    int k = 0;
    uint32_t parity = 0;

    static __host__ __device__ int tensor_bytes(int D, int W) {
        return (32 / W * kHeads * D * (int)sizeof(T) + 127) / 128 * 128;
    }
    static __host__ __device__ size_t warp_bytes(int D, int W) { return (size_t)kAhead * kTensors * tensor_bytes(D, W); }

    __device__ Items(const QkProblem &p, const QkPlan &pl, unsigned char *smem, uint64_t (&bars)[kWarps][kAhead]) {
        const int warp = threadIdx.x / 32;
        bytes = tensor_bytes(p.D, pl.W);
        stage = reinterpret_cast<T *>(smem + warp * warp_bytes(p.D, pl.W));
        full = bars[warp];
        step = gridDim.x * kWarps, step_b = step / pl.tiles, step_tile = step % pl.tiles;
        all = p.B * pl.tiles;
        now.at = (int64_t)blockIdx.x * kWarps + warp;
        now.b = (int)(now.at / pl.tiles), now.tile = (int)(now.at - (int64_t)now.b * pl.tiles);
        next = now;
        if (threadIdx.x % 32 == 0) {
            for (int i = 0; i < kAhead; ++i) tc::mbar_init(full + i, 1);
            tc::fence_mbar_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ T *at(int tensor) const { return stage + (k * kTensors + tensor) * (bytes / (int)sizeof(T)); }
    __device__ __forceinline__ void move(Place &x, const QkPlan &pl) const {
        x.at += step, x.b += step_b, x.tile += step_tile;
        if (x.tile >= pl.tiles) x.tile -= pl.tiles, ++x.b;
    }
    // The next item, into buffer k (skip: a test's that never comes).
    __device__ __forceinline__ void fetch(const QkProblem &p, const QkPlan &pl, const CUtensorMap *const (&maps)[kTensors],
                                          int h0, bool skip = false) {
        if (threadIdx.x % 32 == 0 && next.at < all && !skip) {
            const int t = next.tile * (32 / pl.W);
            int n = 0;
            for (int i = 0; i < kTensors; ++i) n += maps[i] ? 32 / pl.W * kHeads * p.D * (int)sizeof(T) : 0;
            tc::mbar_arrive_expect_tx(full + k, n);
            for (int i = 0; i < kTensors; ++i)
                for (int h = 0; maps[i] && h < kHeads; h += pl.box_heads)
                    for (int d = 0; d < p.D; d += pl.box)
                        tc::tma_load_4d(at(i) + h * p.D + d, maps[i], full + k, d, h0 + h, t, next.b);
        }
        move(next, pl);
    }
    // Waits for buffer k; if it never comes, says so and waits (bounded, too) for all that may be on its way: the shared
    // memory of a CTA that ends is another's.
    __device__ __forceinline__ bool arrived(unsigned int *err) const {
        if (tc::mbar_wait(full + k, parity)) return true;
        atomicOr(err, kDevErrTimeout);
        for (int i = 0; i < kAhead; ++i) tc::mbar_wait(full + (k + i) % kAhead, parity ^ (k + i >= kAhead));
        return false;
    }
    // Done with buffer k: it takes another item, and the warp goes on to its next.
    __device__ __forceinline__ void go_on(const QkProblem &p, const QkPlan &pl, const CUtensorMap *const (&maps)[kTensors],
                                          int h0) {
        __syncwarp();
        fetch(p, pl, maps, h0);
        move(now, pl);
        if (++k == kAhead) k = 0, parity ^= 1;
    }
};

// A lane's token of an item, and its row of the tables (0 where its position is outside of them).
struct Token {
    int64_t at;             // b T + t
    bool in, known;
    int row;
    template <typename I>
    __device__ Token(const QkProblem &p, const QkPlan &pl, const I &items) {
        const int t = items.now.tile * (32 / pl.W) + threadIdx.x % 32 / pl.W;
        in = t < p.T;
        at = in ? items.now.b * p.T + t : 0;
        const int64_t pos = p.R > 0 && p.positions ? (int64_t)p.positions[at] : t;
        known = p.R == 0 || (pos >= 0 && pos < p.P);
        row = known && p.R > 0 ? (int)pos : 0;
    }
};

// The warps of a CTA (blockIdx.x) go over the items, its heads (blockIdx.y) are fixed.
template <typename T, int V, int kHeads, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2)
qk_rows_fwd(const __grid_constant__ QkProblem p, const __grid_constant__ QkMaps maps, const QkPlan pl,
            unsigned int *err) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    using R = typename Pack<T, V>::raw;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bars[kWarps][kAhead];
    const int lane = threadIdx.x % 32, l = lane % pl.W;
    const int which = (int)blockIdx.y >= pl.chunks[0], h0 = ((int)blockIdx.y - (which ? pl.chunks[0] : 0)) * kHeads;
    const QkHeads &hd = p.t[which];
    const Unit<V, kPairs> u(p, l);
    const CUtensorMap *const from[1] = {&maps.x[which]};
    Items<T, 1, kHeads> items(p, pl, smem, bars);
    for (int k = 0; k < kAhead; ++k, ++items.k) items.fetch(p, pl, from, h0, p.stall && k == 0);
    items.k = 0;
    Pairs<V> w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float *from_w = hd.w + u.at[k] + 2 * i;
            w[k][i] = hd.w && u.at[k] >= 0 ? make_float2(__ldg(from_w), __ldg(from_w + 1)) : make_float2(1.f, 1.f);
        }
    Angles<V> angles;
    const float scale = p.norm == 1 ? 1.f / (float)p.D : 1.f;
    for (; items.now.at < items.all; items.go_on(p, pl, from, h0)) {
        const Token tok(p, pl, items);
        const bool turn = u.turn && p.P > 0;
        if (turn) angles.load(p, u.angle, tok.row, false);
        if (!tok.known && tok.in && l == 0) atomicOr(err, kDevErrPages);
        if (!items.arrived(err)) return;
        const T *in = items.at(0) + lane / pl.W * kHeads * p.D;
        const int64_t row = tok.at * hd.heads + h0;
        T *out = static_cast<T *>(hd.out) + row * p.D;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if (h0 + j >= hd.heads) break;              // (the same in the CTA)
            Pairs<V> v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                unpack<T, V>(u.at[k] >= 0 ? *reinterpret_cast<const R *>(in + j * p.D + u.at[k]) : R{}, v[k]);
            float f = 1.f;
            if (p.norm) {
                float2 s2 = tc::mul2(v[0][0], v[0][0]);
#pragma unroll
                for (int i = 1; i < V; ++i) s2 = tc::fma2(v[i / (V / 2)][i % (V / 2)], v[i / (V / 2)][i % (V / 2)], s2);
                const float m = fmaf(scale, sum_lanes(s2.x + s2.y, pl.W), p.eps);
                f = rsqrtf(m);
                // (rare, and decided for the warp: the sum across lanes needs all of them)
                const bool bad = tok.in && !(m >= 1e-30f && m <= 1e37f);
                if (__any_sync(0xffffffffu, bad)) {
                    const float e = m < 1.f ? 0x1p100f : 0x1p-100f;
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float a = v[i / (V / 2)][i % (V / 2)].x * e, d = v[i / (V / 2)][i % (V / 2)].y * e;
                        ss = fmaf(a, a, fmaf(d, d, ss));
                    }
                    ss = sum_lanes(ss, pl.W);
                    if (bad) f = e * rsqrtf(fmaf(scale, ss, p.eps * e * e));
                }
                if (hd.r && tok.in && l == 0) hd.r[row + j] = tok.known ? f : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < V / 2; ++i) v[k][i] = tc::mul2(tc::mul2(v[k][i], make_float2(f, f)), w[k][i]);
            if (turn) angles.template rotate<kPairs>(v[0], v[1]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (tok.in && u.at[k] >= 0)
                    *reinterpret_cast<R *>(out + j * p.D + u.at[k]) = tok.known ? pack<T, V>(v[k]) : R{};
        }
    }
}

// Sums of a CTA's tokens go to part[blockIdx.y][blockIdx.x][D].
template <typename T, int V, int kHeads, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2)
qk_rows_bwd(const __grid_constant__ QkProblem p, const __grid_constant__ QkMaps maps, const QkPlan pl, float *part,
            unsigned int *err) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    using R = typename Pack<T, V>::raw;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t bars[kWarps][kAhead];
    __shared__ float sums[kThreads][V + 1];
    const int lane = threadIdx.x % 32, l = lane % pl.W;
    const int which = (int)blockIdx.y >= pl.chunks[0], h0 = ((int)blockIdx.y - (which ? pl.chunks[0] : 0)) * kHeads;
    const QkHeads &hd = p.t[which];
    const Unit<V, kPairs> u(p, l);
    const CUtensorMap *const from[2] = {&maps.go[which], p.norm ? &maps.x[which] : nullptr};
    Items<T, 2, kHeads> items(p, pl, smem, bars);
    for (int k = 0; k < kAhead; ++k, ++items.k) items.fetch(p, pl, from, h0, p.stall && k == 0);
    items.k = 0;
    Pairs<V> w[2], dw[2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float *from_w = hd.w + u.at[k] + 2 * i;
            w[k][i] = hd.w && u.at[k] >= 0 ? make_float2(__ldg(from_w), __ldg(from_w + 1)) : make_float2(1.f, 1.f);
        }
    Angles<V> angles;
    const float scale = p.norm == 1 ? 1.f / (float)p.D : 1.f;
    for (; items.now.at < items.all; items.go_on(p, pl, from, h0)) {
        const Token tok(p, pl, items);
        const int64_t row = tok.at * hd.heads + h0;
        float f[kHeads];
#pragma unroll
        for (int j = 0; j < kHeads; ++j) f[j] = p.norm && tok.in && h0 + j < hd.heads ? hd.r[row + j] : 1.f;
        const bool turn = u.turn && p.P > 0;
        if (turn) angles.load(p, u.angle, tok.row, true);
        if (!tok.known && tok.in && l == 0) atomicOr(err, kDevErrPages);
        if (!items.arrived(err)) return;
        const int first = lane / pl.W * kHeads * p.D;
        T *out = static_cast<T *>(hd.out) + row * p.D;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if (h0 + j >= hd.heads) break;              // (the same in the CTA)
            Pairs<V> g[2], xh[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = first + j * p.D + u.at[k];
                unpack<T, V>(u.at[k] >= 0 ? *reinterpret_cast<const R *>(items.at(0) + e) : R{}, g[k]);
                unpack<T, V>(u.at[k] >= 0 && p.norm ? *reinterpret_cast<const R *>(items.at(1) + e) : R{}, xh[k]);
            }
            if (turn) angles.template rotate<kPairs>(g[0], g[1]);
            if (p.norm) {
                const float2 f2 = make_float2(f[j], f[j]);
                float2 dots = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        xh[k][i] = tc::mul2(xh[k][i], f2);
                        const float2 gx = tc::mul2(g[k][i], xh[k][i]);
                        if (tok.in && tok.known) dw[k][i] = tc::add2(dw[k][i], gx);
                        dots = tc::fma2(gx, w[k][i], dots);
                    }
                const float dot = -sum_lanes(dots.x + dots.y, pl.W) * scale;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < V / 2; ++i)
                        g[k][i] = tc::mul2(f2, tc::fma2(xh[k][i], make_float2(dot, dot), tc::mul2(g[k][i], w[k][i])));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (tok.in && u.at[k] >= 0)
                    *reinterpret_cast<R *>(out + j * p.D + u.at[k]) = tok.known ? pack<T, V>(g[k]) : R{};
        }
    }
    if (!part) return;
    // the segments of the CTA are added in their order
    float *to = part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * p.D;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) sums[threadIdx.x][i] = i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x;
        __syncthreads();
        for (int e = threadIdx.x; e < pl.W * V; e += kThreads) {
            const Unit<V, kPairs> o(p, e / V);
            if (o.at[j] < 0) continue;
            float s = 0.f;
            for (int r = 0; r < kThreads / pl.W; ++r) s += sums[r * pl.W + e / V][e % V];
            to[o.at[j] + e % V] = s;
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
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    __shared__ float rows[32][33];
    const int which = blockIdx.y, col = threadIdx.x % 32, row = threadIdx.x / 32, i = blockIdx.x * 32 + col;
    float s = 0.f;
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
    if (p.D > 256 && p.D % 128 != 0) return false;      // (two boxes, each from 128 bytes of shared memory on)
    if (std::max(p.t[0].heads, p.t[1].heads) > 30000) return false;     // (grid y)
    if (p.R > 0 && (!on16(p.cos) || !on16(p.sin))) return false;
    for (const QkHeads &t : p.t) {
        if (t.heads == 0) continue;
        // (strides that a tensor map holds)
        const int64_t wide = int64_t(1) << 38;
        if (!on16(t.x) || t.x_b * es % 16 || t.x_t * es % 16 || t.x_h * es % 16) return false;
        if (t.go && (!on16(t.go) || t.g_b * es % 16 || t.g_t * es % 16 || t.g_h * es % 16)) return false;
        if (std::max({t.x_b, t.x_t, t.x_h}) >= wide || (t.go && std::max({t.g_b, t.g_t, t.g_h}) >= wide)) return false;
    }
    return true;
}

QkPlan plan_of(const QkProblem &p, int heads) {
    const int V = p.io == 0 ? 8 : 4, units = (p.D + 2 * V - 1) / (2 * V);
    QkPlan pl;
    pl.W = 1;
    while (pl.W < units) pl.W *= 2;
    const int per = std::max(1, 32 / pl.W);
    for (int i = 0; i < 2; ++i) pl.chunks[i] = (p.t[i].heads + heads - 1) / heads;
    pl.tiles = (int)((p.T + per - 1) / per);
    // (a box holds at most 256 values of a row)
    pl.box = p.D <= 256 ? p.D : p.D / 2;
    pl.box_heads = p.D <= 256 ? heads : 1;
    return pl;
}
// CTAs over the items: one round of resident ones (two to an SM), or a warp for each item.
unsigned item_ctas(const QkProblem &p, const QkPlan &pl, int num_sms) {
    const int64_t need = (p.B * pl.tiles + kWarps - 1) / kWarps;
    const int64_t most = std::max(1, 2 * num_sms / std::max(1, pl.chunks[0] + pl.chunks[1]));
    return (unsigned)std::min(need, most);
}
// One sequence for many, where their rows follow each other: items then end inside of none (a token of each of many rows
// is one sequence). Without positions of its own a token's place in its sequence is its position.
QkProblem joined(QkProblem p) {
    bool row = p.B > 1 && (p.positions || p.R == 0) && p.B * p.T < int64_t(1) << 30;
    for (const QkHeads &t : p.t)
        if (t.heads > 0 && p.T > 1 && (t.x_b != p.T * t.x_t || (t.go && t.g_b != p.T * t.g_t))) row = false;
    if (!row) return p;
    if (p.T == 1)
        for (QkHeads &t : p.t) t.x_t = t.x_b, t.g_t = t.g_b;
    p.T *= p.B;
    p.B = 1;
    for (QkHeads &t : p.t) t.x_b = p.T * t.x_t, t.g_b = p.T * t.g_t;
    return p;
}

bool make_map(CUtensorMap *m, const void *base, const QkProblem &p, const QkPlan &pl, int heads, int64_t sb, int64_t st,
              int64_t sh) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t es = p.io == 0 ? 2 : 4;
    const cuuint64_t dims[4] = {(cuuint64_t)p.D, (cuuint64_t)heads, (cuuint64_t)p.T, (cuuint64_t)p.B};
    const cuuint64_t strides[3] = {(cuuint64_t)sh * es, (cuuint64_t)st * es, (cuuint64_t)sb * es};
    const cuuint32_t box[4] = {(cuuint32_t)pl.box, (cuuint32_t)pl.box_heads, (cuuint32_t)(32 / pl.W), 1}, one[4] = {1, 1, 1, 1};
    return fn(m, p.io == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
              const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool make_maps(const QkProblem &p, const QkPlan &pl, QkMaps *m) {
    for (int i = 0; i < 2; ++i) {
        const QkHeads &t = p.t[i];
        if (t.heads == 0) continue;
        if (!make_map(&m->x[i], t.x, p, pl, t.heads, t.x_b, t.x_t, t.x_h)) return false;
        if (t.go && !make_map(&m->go[i], t.go, p, pl, t.heads, t.g_b, t.g_t, t.g_h)) return false;
    }
    return true;
}

template <typename T, bool kPairs>
cudaError_t rows_fwd(const QkProblem &p, int num_sms, unsigned int *err, cudaStream_t s) {
    constexpr auto kernel = qk_rows_fwd<T, 16 / sizeof(T), kFwdHeads, kPairs>;
    const QkPlan pl = plan_of(p, kFwdHeads);
    QkMaps maps;
    if (!make_maps(p, pl, &maps)) return cudaErrorInvalidResourceHandle;
    const size_t smem = kWarps * Items<T, 1, kFwdHeads>::warp_bytes(p.D, pl.W);
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    return launch(kernel, dim3(item_ctas(p, pl, num_sms), pl.chunks[0] + pl.chunks[1]), kThreads, smem, s, p, maps, pl,
                  err);
}
template <typename T, bool kPairs>
cudaError_t rows_bwd(const QkProblem &p, float *part, int num_sms, unsigned int *err, cudaStream_t s, QkSums *sums) {
    constexpr auto kernel = qk_rows_bwd<T, 16 / sizeof(T), kBwdHeads, kPairs>;
    const QkPlan pl = plan_of(p, kBwdHeads);
    QkMaps maps;
    if (!make_maps(p, pl, &maps)) return cudaErrorInvalidResourceHandle;
    const dim3 grid(item_ctas(p, pl, num_sms), pl.chunks[0] + pl.chunks[1]);
    const size_t smem = kWarps * Items<T, 2, kBwdHeads>::warp_bytes(p.D, pl.W);
    for (int i = 0; i < 2; ++i) {
        sums->part[i] = part + (i ? (size_t)pl.chunks[0] * grid.x * p.D : 0);
        sums->n[i] = (int64_t)pl.chunks[i] * grid.x;
        sums->stride[i] = p.D;
    }
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    return launch(kernel, grid, kThreads, smem, s, p, maps, pl, part, err);
}

template <typename T>
cudaError_t run_fwd(const QkProblem &in, int num_sms, unsigned int *err, cudaStream_t s) {
    if (!vectors(in))
        return launch(qk_plain_fwd<T>, dim3((unsigned)((rows_of(in) + kWarps - 1) / kWarps)), kThreads, 0, s, in,
                      err);
    QkProblem p = joined(in);
    p.stall = take_stall_hook();
    return p.pairs ? rows_fwd<T, true>(p, num_sms, err, s) : rows_fwd<T, false>(p, num_sms, err, s);
}

template <typename T>
cudaError_t run_bwd(const QkProblem &in, float *part, int num_sms, unsigned int *err, cudaStream_t s) {
    QkSums sums{};
    cudaError_t e;
    if (vectors(in)) {
        QkProblem p = joined(in);
        p.stall = take_stall_hook();
        e = p.pairs ? rows_bwd<T, true>(p, part, num_sms, err, s, &sums) : rows_bwd<T, false>(p, part, num_sms, err, s, &sums);
    } else {
        constexpr auto kernel = qk_plain_bwd<T>;
        const int parts = bwd_parts(in, num_sms);
        const size_t smem = 2 * kWarps * (size_t)in.D * sizeof(float);
        for (int i = 0; i < 2; ++i) {
            sums.part[i] = part + (i ? in.D : 0);
            sums.n[i] = parts;
            sums.stride[i] = 2 * in.D;
        }
        e = allow_shared<kernel>();
        if (e != cudaSuccess) return e;
        e = launch(kernel, dim3(parts), kThreads, smem, s, in, part, err);
    }
    if (e != cudaSuccess || !part) return e;
    return launch(qk_sums_kernel, dim3((in.D + 31) / 32, 2), 1024, 0, s, in, sums);
}

}  // namespace

cudaError_t launch_qk_fwd(const QkProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    return p.io == 0 ? run_fwd<__nv_bfloat16>(p, num_sms, dev_err, s) : run_fwd<float>(p, num_sms, dev_err, s);
}

// (what either kernel needs: the one that runs depends on the pointers)
size_t qk_bwd_workspace_bytes(const QkProblem &p, int num_sms) {
    if (!p.norm) return 0;
    const QkPlan pl = plan_of(p, kBwdHeads);
    // (sequences that a call joins have no more items than they have apart)
    const size_t plain = (size_t)bwd_parts(p, num_sms) * 2,
                 vec = pl.W > 32 ? 0 : (size_t)item_ctas(p, pl, num_sms) * (pl.chunks[0] + pl.chunks[1]);
    return std::max(plain, vec) * p.D * sizeof(float);
}

cudaError_t launch_qk_bwd(const QkProblem &p, void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    float *part = p.norm && (p.t[0].dw || p.t[1].dw) ? static_cast<float *>(ws) : nullptr;
    return p.io == 0 ? run_bwd<__nv_bfloat16>(p, part, num_sms, dev_err, s)
                     : run_bwd<float>(p, part, num_sms, dev_err, s);
}

}  // namespace gla
