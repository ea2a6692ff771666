// Selective state space scan: N states per channel, whose decays are inputs,
//     h_t = a_t h_{t-1} + d_t u_t B_t,   a_t = e^(d_t A),   y_t = C_t . h_t + D u_t,   o_t = y_t silu(z_t)
// and its gradients. With dy = d_o silu(z), G_t the gradient of h_t and G'_t = a_t G_t what it passes
// to the token before:
//     G_t = C_t dy_t + G'_{t+1},   w_t = G'_t h_{t-1}
//     dd_t = sum_n w_t A + u_t sum_n G_t B_t,   du_t = d_t sum_n G_t B_t + D dy_t
//     dA = sum_t w_t d_t,   dB_t = sum_c G_t d_t u_t,   dC_t = sum_c h_t dy_t
//
// A ring of warps: a CTA owns 32 kCh channels of a sequence (kCh to a lane), and its warps take chunks of
// kTok tokens in turn, four states of a lane at a time. All that a chunk can do without the state
// (loads, step sizes, exponentials, inputs) runs while the chunks before it are still at work; the
// states then come from the warp before through shared memory, walk over the chunk's tokens in registers
// and go on to the next warp. So a sequence is walked once and each exponential is computed once,
// although all warps work at the same time. Backwards the ring turns the other way, on the states
// that a forward walk left at the start of each chunk.
//
// Pairs of packed arithmetic are two tokens of one state: step sizes, inputs, B, C and sums of outputs
// then are pairs as they come, and only the walk itself is scalar. (Pairs of two states need each
// token's d and d u twice, which cost more moves than the walk saved: 191 instructions for a
// token and channel of 16 states.)
//
// Bound: 16 exponentials of a token and channel take 64 cycles of a scheduler's share of the special function
// units, the four multiply-adds of each state 64 of its FP32 pipe; in the backward pass thirteen of them 208.
#include <cuda_bf16.h>

#include <algorithm>
#include <stdlib.h>

#include "elem.cuh"
#include "gla_internal.h"
#include "ssm.h"
#include "tma_host.h"

namespace gla {
namespace {

constexpr int kTok = 8;             // tokens of a chunk
constexpr int kPairs = kTok / 2;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

using tc::add2;
using tc::fma2;
using tc::mul2;
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 2^(A d) of a pair of tokens. The hardware's 2^x is good to 1.2e-7 but lies low on average, by up to 2.6e-8 of
// the value for x in (-1/8, 0): over the hundred tokens that such decays remember this adds up, to 4e-6 of
// the state. 2e-8 on the exponent's side (which costs nothing, as the product is a multiply-add) leaves at
// most 1.3e-8 on average, a quarter of fp32's rounding; 2^0 is still 1.
__device__ __forceinline__ float2 decay2(float2 A, float2 d) {
    const float2 x = fma2(A, d, both(2e-8f));
    return make_float2(ex2(x.x), ex2(x.y));
}

// A times log2 e, with infinities brought to the largest float: a step of zero then keeps the state.
__device__ __forceinline__ float scale_a(float a) {
    const float x = a * kLog2e;
    return isinf(x) ? copysignf(3.4028235e38f, x) : x;
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x|. log(1 + e) is e times a polynomial fitted to
// log(1 + e) / e on [0, 1] with the smallest relative error (5e-9, 1.4e-7 with the roundings of fp32): the
// small steps that give a state its memory keep their digits, which log(1 + e) formed as such would lose, and
// ten multiply-adds cost a third of the library's functions. (Scalar: packed ones would have to fetch
// their constants into registers.)
__device__ __forceinline__ float softplus(float x) {
    const float e = ex2(fabsf(x) * -kLog2e);
    float r = -0.003244024235755205f;
    r = fmaf(r, e, 0.019851457327604294f);
    r = fmaf(r, e, -0.056959524750709534f);
    r = fmaf(r, e, 0.10603654384613037f);
    r = fmaf(r, e, -0.15305592119693756f);
    r = fmaf(r, e, 0.1967593878507614f);
    r = fmaf(r, e, -0.24954134225845337f);
    r = fmaf(r, e, 0.3332996368408203f);
    r = fmaf(r, e, -0.4999990165233612f);
    r = fmaf(r, e, 1.f);
    return fmaf(r, e, fmaxf(x, 0.f));
}
__device__ __forceinline__ float step_size(float x, int on) { return on ? softplus(x) : x; }

// What a CTA's warps read: the sequence's rows from the tile's first channel (the group's B and C) on.
struct Source {
    const void *p;
    int64_t t;          // element stride of a token
    int width;          // elements that exist, of a row of `row` in the stage
    int row;
};

// Brings the tokens [t0, t0 + kTok) of a source into to[kTok][row] element by element, with zeros for tokens and
// elements that do not exist: what TMA does where rows are on 16 bytes.
template <typename T>
__device__ __forceinline__ void stage_rows(const Source &s, int64_t t0, int64_t T_, T *to) {
    const T *p = static_cast<const T *>(s.p) + t0 * s.t;
    T zero;
    put(&zero, 0.f);
    for (int k = threadIdx.x % 32; k < kTok * s.row; k += 32) {
        const int i = k / s.row, v = k - i * s.row;
        to[k] = t0 + i < T_ && v < s.width ? p[i * s.t + v] : zero;
    }
}

// Tensor maps of the rows: boxes of kTok tokens by a tile's channels (or a group's states).
struct Maps {
    CUtensorMap in[4], b, c, out[3];
};

// B and C of the chunk as floats, the values of two tokens side by side as the packed arithmetic takes
// them: from[2][kTok][N] -> to[2][kTok / 2][NP] float2, NP = N up to a multiple of 4, zero past N.
template <typename T, int kN>
__device__ __forceinline__ void widen_rows(const T *from, float2 *to, int N) {
    const int lane = threadIdx.x % 32, NP = (N + 3) / 4 * 4;
    if constexpr (kN > 0) {     // four states at a time
#pragma unroll
        for (int k = lane; k < kTok * kN / 4; k += 32) {
            const int row = k / (kN / 4), q = k % (kN / 4);     // row: a pair of tokens of B, or of C
            float x[4], y[4];
            Pack<T, 4>::unpack(*reinterpret_cast<const typename Pack<T, 4>::raw *>(from + 2 * row * N + 4 * q), x);
            Pack<T, 4>::unpack(*reinterpret_cast<const typename Pack<T, 4>::raw *>(from + (2 * row + 1) * N + 4 * q), y);
            float4 *t = reinterpret_cast<float4 *>(to + row * NP + 4 * q);
            t[0] = make_float4(x[0], y[0], x[1], y[1]);
            t[1] = make_float4(x[2], y[2], x[3], y[3]);
        }
    } else {
        for (int k = lane; k < kTok * NP; k += 32) {
            const int row = k / NP, n = k - row * NP;
            to[k] = n < N ? make_float2(get(from + 2 * row * N + n), get(from + (2 * row + 1) * N + n)) : both(0.f);
        }
    }
}

// Hand-overs. Addresses are those of shared memory, so that a step's are immediate offsets of a chunk's.
struct Link {
    uint32_t bar, slot;             // step 0 of a warp (32 slots of 16 bytes and one barrier to a step)
};
__device__ __forceinline__ float4 load4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store4(uint32_t at, const float (&v)[4]) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Most hand-overs arrive while it polls; the clock that bounds the wait takes longer to read than they do. A warp that
// gave up once (dead) does not wait again.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, bool dead, unsigned int *err) {
    if (dead) return true;
#pragma unroll 1
    for (int i = 0; i < 256; ++i)
        if (try_wait(bar, parity)) return false;
    const uint64_t t0 = tc::global_ns();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (try_wait(bar, parity)) return false;
        if (tc::global_ns() - t0 > tc::kWaitLimitNs) break;
    }
    atomicOr(err, kDevErrTimeout);
    return true;
}
// Lane 0 tells the next warp, once all lanes have written.
__device__ __forceinline__ void hand_over(uint32_t bar, int lane) {
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 st;\n\t"
        "setp.eq.s32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.release.cta.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar), "r"(lane)
        : "memory");
}

// The CTAs of a sequence: tiles of 32 kCh channels of one group.
struct Tiles {
    int per_group;
    int64_t all;
};
__host__ __device__ inline Tiles tiles_of(int64_t C, int64_t G, int ch) {
    const int64_t n = (C / G + 32 * ch - 1) / (32 * ch);
    return Tiles{(int)n, n * G};
}

// Segments of a sequence: with few channels it is cut, so that all SMs have a part. The segments' states from zero come
// first, then those that they start from (ssm_join_kernel), then the walk over all segments at once.
struct Split {
    int n;                          // segments of a sequence
    int64_t chunks;                 // of each but the last
    float *h, *g;                   // [B][n][C][N]: what a segment ends with if it starts from zero, then what it
                                    // starts from (g: backwards)
    float *sum;                     // [B][n][C]: the segment's step sizes
};

// Where a CTA is: a sequence (a segment of it), a group of channels and 32 kCh of them.
template <int kCh>
struct Place {
    int64_t b, row, tile, g, c0;    // row: b n + the segment; c0: the first channel
    int seg;
    int64_t ch0, ch1;               // chunks
    int width, mine;                // channels of the tile, of the lane
    __device__ Place(const SsmProblem &p, const Tiles &tl, const Split &sp, int segs) {
        tile = blockIdx.x % tl.all;
        const int64_t i = blockIdx.x / tl.all;
        b = i / segs;
        seg = (int)(i - b * segs);
        row = b * sp.n + seg;
        ch0 = seg * sp.chunks;
        ch1 = min(ch0 + sp.chunks, (p.T + kTok - 1) / kTok);
        g = tile / tl.per_group;
        const int64_t cg = p.C / p.G, first = (tile - g * tl.per_group) * 32 * kCh;
        width = (int)min((int64_t)32 * kCh, cg - first);
        c0 = g * cg + first;
        mine = max(0, min(kCh, width - kCh * (int)(threadIdx.x % 32)));
    }
    // Channel j of the lane; the tile's first one where there is none.
    __device__ int64_t channel(int j) const { return c0 + (j < mine ? threadIdx.x % 32 * kCh + j : 0); }
    template <typename T>
    __device__ Source channels(const SsmRows &r) const {
        return Source{r.p ? static_cast<const T *>(r.p) + b * r.b + c0 : nullptr, r.t, width, 32 * kCh};
    }
    template <typename T>
    __device__ Source rows(const SsmRows &r, int N) const {
        return Source{static_cast<const T *>(r.p) + b * r.b + g * N, r.t, N, N};
    }
};

// States [kCh][kSt] of step q of the lane, from and to row `row` of [rows, C, N].
template <int kCh>
__device__ __forceinline__ void load_states(const float *from, int64_t row, const SsmProblem &p, const Place<kCh> &at,
                                            int q, float (&h)[4]) {
    constexpr int kSt = 4 / kCh;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = kSt * q + j % kSt;
        h[j] = from && j / kSt < at.mine && n < p.N ? from[(row * p.C + at.channel(j / kSt)) * p.N + n] : 0.f;
    }
}
template <int kCh>
__device__ __forceinline__ void store_states(float *to, int64_t row, const SsmProblem &p, const Place<kCh> &at,
                                             int q, const float (&h)[4]) {
    constexpr int kSt = 4 / kCh;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int n = kSt * q + j % kSt;
        if (j / kSt < at.mine && n < p.N) to[(row * p.C + at.channel(j / kSt)) * p.N + n] = h[j];
    }
}

// A lane works on kSt = 4 / kCh states of its channels at a time, Q = N / kSt times. Shared memory of a
// ring of W warps:
//   slot[W][Q][32] float4: what a warp hands on, [kCh][kSt];  A[Q][2][32] float4: A log2 e, twice each
//   sums[W][Q][32] float4 (backward): dA;  turn[W][32][kTurn] float (backward): sums across lanes
//   rows[W][2][kPairs][NP] float2: B and C of a warp's chunk;  bar[W][Q]
//   stage[W][2]: a chunk as it lies in memory, on its way while the one before it is worked on:
//     kIn tensors [kTok][32 kCh], then B and C [kTok][N];  full[W][2]: it is there
//   dx[W][kPairs][kCh][32] float4 (forward): d and d u of a warp's chunk
constexpr int kTurn = 66;           // (lanes that write pairs side by side meet no bank twice)
template <typename T, int kCh>
struct Ring {
    float4 *slot, *A, *sums;
    float *turn;
    float2 *rows;
    uint64_t *bar, *full;
    unsigned char *stage;
    static __host__ __device__ int steps(int N) { return (N + 4 / kCh - 1) / (4 / kCh); }
    static __host__ __device__ int padded(int N) { return (N + 3) / 4 * 4; }
    static __host__ __device__ size_t stage_bytes(int in, int N) {
        return ((size_t)in * kTok * 32 * kCh * sizeof(T) + 2 * kTok * (size_t)N * sizeof(T) + 127) / 128 * 128;
    }
    static __host__ __device__ size_t round(size_t n) { return (n + 127) / 128 * 128; }
    static __host__ __device__ size_t stage_at(int W, int N, bool backward) {
        const size_t Q = steps(N);
        return W * Q * 32 * 16 * (backward ? 2 : 1) + Q * 2 * 32 * 16 + (backward ? round(W * 32 * kTurn * 4) : 0) +
               round((size_t)W * 2 * kPairs * padded(N) * 8) + round(W * (Q + 2) * 8);
    }
    static __host__ __device__ size_t bytes(int W, int in, int N, bool backward) {
        return stage_at(W, N, backward) + 2 * W * stage_bytes(in, N) + (backward ? 0 : W * kPairs * kCh * 32 * 16);
    }
    __device__ Ring(unsigned char *smem, int W, int N, bool backward) {
        const int Q = steps(N);
        slot = reinterpret_cast<float4 *>(smem);
        A = slot + W * Q * 32;
        sums = A + Q * 2 * 32;
        turn = reinterpret_cast<float *>(sums + (backward ? W * Q * 32 : 0));
        rows = reinterpret_cast<float2 *>(reinterpret_cast<unsigned char *>(turn) + (backward ? round(W * 32 * kTurn * 4) : 0));
        bar = reinterpret_cast<uint64_t *>(reinterpret_cast<unsigned char *>(rows) + round((size_t)W * 2 * kPairs * padded(N) * 8));
        full = bar + W * Q;
        stage = smem + stage_at(W, N, backward);
    }
    // A, the barriers, and the states that the first chunk takes over, as if from the last warp; the CTA synchronises.
    __device__ void begin(const SsmProblem &p, const Place<kCh> &at, int W, int N, const float *first, int64_t row) {
        constexpr int kSt = 4 / kCh;
        const int Q = steps(N), lane = threadIdx.x % 32;
        for (int q = threadIdx.x / 32; q < Q; q += W) {
            float a[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = kSt * q + j % kSt;
                a[j] = n < N && j / kSt < at.mine ? scale_a(p.A[at.channel(j / kSt) * N + n]) : 0.f;
            }
            A[2 * q * 32 + lane] = make_float4(a[0], a[0], a[1], a[1]);
            A[(2 * q + 1) * 32 + lane] = make_float4(a[2], a[2], a[3], a[3]);
            load_states<kCh>(first, row, p, at, q, a);
            slot[((W - 1) * Q + q) * 32 + lane] = make_float4(a[0], a[1], a[2], a[3]);
        }
        if (threadIdx.x == 0) {
            for (int i = 0; i < W * (Q + 2); ++i) tc::mbar_init(bar + i, 1);
            tc::fence_mbar_init();
        }
        __syncthreads();
        for (int q = threadIdx.x; q < Q; q += 32 * W) tc::mbar_arrive(bar + (W - 1) * Q + q);
    }
    __device__ Link link(int w, int Q) const {
        return Link{tc::smem_u32(bar + w * Q), tc::smem_u32(slot + w * Q * 32 + threadIdx.x % 32)};
    }
    __device__ void load_a(int q, float2 (&a)[4]) const {
        const int lane = threadIdx.x % 32;
        const float4 x = A[2 * q * 32 + lane], y = A[(2 * q + 1) * 32 + lane];
        a[0] = make_float2(x.x, x.y);
        a[1] = make_float2(x.z, x.w);
        a[2] = make_float2(y.x, y.y);
        a[3] = make_float2(y.z, y.w);
    }
};

// The lane's channels of row i of a tensor in the stage.
template <typename T, int kCh>
__device__ __forceinline__ void lane_row(const T *in, int i, float (&v)[kCh]) {
    const T *r = in + (i * 32 + threadIdx.x % 32) * kCh;
    if constexpr (kCh == 1) {
        v[0] = get(r);
    } else if constexpr (sizeof(T) == 2) {
        const float2 f = tc::unpack_bf16(*reinterpret_cast<const uint32_t *>(r));
        v[0] = f.x;
        v[1] = f.y;
    } else {
        const float2 f = *reinterpret_cast<const float2 *>(r);
        v[0] = f.x;
        v[1] = f.y;
    }
}
template <typename T, int kCh>
__device__ __forceinline__ void put_lane_row(T *to, int i, const float (&v)[kCh]) {
    T *r = to + (i * 32 + threadIdx.x % 32) * kCh;
    if constexpr (kCh == 1) {
        put(r, v[0]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint32_t *>(r) = tc::pack_bf16(v[0], v[1]);
    } else {
        *reinterpret_cast<float2 *>(r) = make_float2(v[0], v[1]);
    }
}
// The same for a pair of tokens: v[channel] = (token 2 ip, token 2 ip + 1).
template <typename T, int kCh>
__device__ __forceinline__ void lane_pair(const T *in, int ip, float2 (&v)[kCh]) {
    float x[kCh], y[kCh];
    lane_row<T, kCh>(in, 2 * ip, x);
    lane_row<T, kCh>(in, 2 * ip + 1, y);
#pragma unroll
    for (int c = 0; c < kCh; ++c) v[c] = make_float2(x[c], y[c]);
}
template <typename T, int kCh>
__device__ __forceinline__ void put_lane_pair(T *to, int ip, const float2 (&v)[kCh]) {
    float x[kCh], y[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        x[c] = v[c].x;
        y[c] = v[c].y;
    }
    put_lane_row<T, kCh>(to, 2 * ip, x);
    put_lane_row<T, kCh>(to, 2 * ip + 1, y);
}
// Rows of the stage to the tile's rows of a contiguous [B, T, C] tensor, where TMA does not do it.
template <typename T, int kCh>
__device__ __forceinline__ void write_rows(const T *from, void *to, const SsmProblem &p, const Place<kCh> &at, int64_t t0) {
    T *out = static_cast<T *>(to) + (at.b * p.T + t0) * p.C + at.c0;
    for (int i = 0; i < kTok; ++i)
        for (int v = threadIdx.x % 32; v < at.width; v += 32)
            if (t0 + i < p.T) out[i * p.C + v] = from[i * 32 * kCh + v];
}

// Step sizes of the chunk from the stage (zero for tokens and channels that do not exist: they keep the state).
template <typename T, int kCh>
__device__ __forceinline__ void step_sizes(const T *in, const float (&bias)[kCh], int plus, int64_t left, int mine,
                                           float2 (&d)[kCh][kPairs]) {
#pragma unroll
    for (int ip = 0; ip < kPairs; ++ip) {
        float2 r[kCh];
        lane_pair<T, kCh>(in, ip, r);
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
            d[c][ip] = add2(r[c], both(bias[c]));
        }
    }
    if (plus) {
#pragma unroll
        for (int c = 0; c < kCh; ++c)
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) d[c][ip] = make_float2(softplus(d[c][ip].x), softplus(d[c][ip].y));
    }
    if (left < kTok || mine < kCh) {
#pragma unroll
        for (int c = 0; c < kCh; ++c)
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                if (c >= mine || 2 * ip >= left) d[c][ip].x = 0.f;
                if (c >= mine || 2 * ip + 1 >= left) d[c][ip].y = 0.f;
            }
    }
}

// Two states' pairs of row ip of B (or C).
template <int kSt>
__device__ __forceinline__ void load_bc(const float2 *row, int q, float2 (&v)[kSt]) {
#pragma unroll
    for (int n = 0; n < kSt; n += 2) {
        const float4 x = *reinterpret_cast<const float4 *>(row + kSt * q + n);
        v[n] = make_float2(x.x, x.y);
        v[n + 1] = make_float2(x.z, x.w);
    }
}

// What a forward walk leaves: outputs and the last state; the states before each chunk (marks
// [B][chunks][tiles][Q][32] float4), which the backward walk needs; a segment's last state and step sizes (Split).
enum { kOutputs = 0, kMarks = 1, kEnds = 2 };

// kN: N, if known at compile time. segs: segments of a sequence that this call walks over.
template <typename T, int kCh, int kN, int kMode, bool kVec>
__global__ void __launch_bounds__(512, 1)
ssm_fwd_kernel(const __grid_constant__ SsmProblem p, const __grid_constant__ Maps maps, const Split sp, int segs,
               float4 *marks, unsigned int *err) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float sums[kMode == kEnds ? 16 : 1][32 * kCh];
    constexpr bool kOut = kMode == kOutputs;
    constexpr int kSt = 4 / kCh, kIn = kOut ? 3 : 2, kRow = kTok * 32 * kCh;
    using R = Ring<T, kCh>;
    const int W = blockDim.x / 32, N = kN ? kN : p.N, Q = R::steps(N), NP = R::padded(N);
    R ring(smem, W, N, false);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G, kCh);
    const Place<kCh> at(p, tl, sp, segs);
    ring.begin(p, at, W, N, kMode == kEnds ? nullptr : sp.n > 1 ? sp.h : p.h0, sp.n > 1 ? at.row : at.b);
    float bias[kCh], D[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        bias[c] = p.dt_bias ? p.dt_bias[at.channel(c)] : 0.f;
        D[c] = p.D ? p.D[at.channel(c)] : 0.f;
    }
    float2 *rows = ring.rows + w * 2 * kPairs * NP;
    const size_t stage_bytes = R::stage_bytes(kIn, N);
    auto stage = [&](int k) { return reinterpret_cast<T *>(ring.stage + (2 * w + k) * stage_bytes); };
    // d and d u of a chunk: in registers they would cost a tenth more instructions (moves; 128 registers are few)
    float4 *dx = reinterpret_cast<float4 *>(ring.stage + 2 * W * stage_bytes) + w * kPairs * kCh * 32 + lane;
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    // the chunk into buffer k of the stage, by one lane where TMA does it
    auto fetch = [&](int64_t ch, int k) {
        if (ch >= at.ch1) return;
        T *to = stage(k);
        const int64_t t0 = ch * kTok;
        if (kVec) {
            if (lane == 0) {
                uint64_t *bar = ring.full + 2 * w + k;
                const bool z = kOut && p.z.p;
                tc::bulk_wait_read_all();       // the outputs that were there
                tc::mbar_arrive_expect_tx(bar, ((z ? 3 : 2) * kRow + 2 * kTok * N) * (int)sizeof(T));
                const int c = (int)at.c0, b = (int)at.b, t = (int)t0, n = (int)at.g * N;
                tc::tma_load_4d(to, &maps.in[0], bar, c, t, b, 0);
                tc::tma_load_4d(to + kRow, &maps.in[1], bar, c, t, b, 0);
                if (z) tc::tma_load_4d(to + 2 * kRow, &maps.in[2], bar, c, t, b, 0);
                tc::tma_load_4d(to + kIn * kRow, &maps.b, bar, n, t, b, 0);
                tc::tma_load_4d(to + kIn * kRow + kTok * N, &maps.c, bar, n, t, b, 0);
            }
        } else {
            stage_rows<T>(at.template channels<T>(p.u), t0, p.T, to);
            stage_rows<T>(at.template channels<T>(p.dt), t0, p.T, to + kRow);
            if (kOut && p.z.p) stage_rows<T>(at.template channels<T>(p.z), t0, p.T, to + 2 * kRow);
            stage_rows<T>(at.template rows<T>(p.Bm, N), t0, p.T, to + kIn * kRow);
            stage_rows<T>(at.template rows<T>(p.Cm, N), t0, p.T, to + kIn * kRow + kTok * N);
        }
    };
    const Link from = ring.link(w == 0 ? W - 1 : w - 1, Q), to = ring.link(w, Q);
    const uint32_t full = tc::smem_u32(ring.full + 2 * w);
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!try_wait(bar, parity)) dead = wait_on(bar, parity, dead, err);
    };
    int k = 0;
    uint32_t round = 0, parity = 0;     // of the stage's buffer, and of the hand-overs
    float2 total[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) total[c] = both(0.f);
    fetch(at.ch0 + w, 0);
    for (int64_t ch = at.ch0 + w; ch < at.ch1; ch += W) {
        const int64_t t0 = ch * kTok;
        if (kVec) wait(full + 8 * k, round);
        else __syncwarp();
        T *in = stage(k);
        widen_rows<T, kN>(in + kIn * kRow, rows, N);
        float2 d[kCh][kPairs], y[kCh][kPairs];
        step_sizes<T, kCh>(in + kRow, bias, p.softplus, p.T - t0, at.mine, d);
#pragma unroll
        for (int ip = 0; ip < kPairs; ++ip) {
            float2 u[kCh];
            lane_pair<T, kCh>(in, ip, u);
#pragma unroll
            for (int c = 0; c < kCh; ++c) {
                const float2 x = c < at.mine ? mul2(d[c][ip], u[c]) : both(0.f);
                dx[(ip * kCh + c) * 32] = make_float4(d[c][ip].x, d[c][ip].y, x.x, x.y);
                y[c][ip] = both(0.f);
                if (kMode == kEnds) total[c] = add2(total[c], d[c][ip]);
            }
        }
        __syncwarp();
        fetch(ch + W, k ^ 1);
#pragma unroll 1
        for (int q = 0; q < Q; ++q) {
            float2 A[4], a[4][kPairs], s[4][kPairs];      // [kCh][kSt]
            ring.load_a(q, A);
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                float2 b[kSt];
                load_bc<kSt>(rows + ip * NP, q, b);
                float4 v[kCh];
#pragma unroll
                for (int c = 0; c < kCh; ++c) v[c] = dx[(ip * kCh + c) * 32];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j][ip] = decay2(A[j], make_float2(v[j / kSt].x, v[j / kSt].y));
                    s[j][ip] = mul2(b[j % kSt], make_float2(v[j / kSt].z, v[j / kSt].w));
                }
            }
            wait(from.bar + 8 * q, parity);
            const float4 v = load4(from.slot + 512 * q);
            float h[4] = {v.x, v.y, v.z, v.w};
            if (kMode == kMarks)
                marks[(((at.b * chunks + ch) * tl.all + at.tile) * Q + q) * 32 + lane] = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[j][ip].x = fmaf(a[j][ip].x, h[j], s[j][ip].x);
                    h[j] = s[j][ip].y = fmaf(a[j][ip].y, s[j][ip].x, s[j][ip].y);
                }
            store4(to.slot + 512 * q, h);
            hand_over(to.bar + 8 * q, lane);
            if (kOut) {
#pragma unroll
                for (int ip = 0; ip < kPairs; ++ip) {
                    float2 c[kSt];
                    load_bc<kSt>(rows + (kPairs + ip) * NP, q, c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j / kSt][ip] = fma2(c[j % kSt], s[j][ip], y[j / kSt][ip]);
                }
            }
        }
        if (kOut) {
            // outputs take the place of u in the stage, then leave in whole rows
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                float2 u[kCh], z[kCh];
                if (p.D) lane_pair<T, kCh>(in, ip, u);
                if (p.z.p) lane_pair<T, kCh>(in + 2 * kRow, ip, z);
#pragma unroll
                for (int c = 0; c < kCh; ++c) {
                    if (p.D) y[c][ip] = fma2(both(D[c]), u[c], y[c][ip]);
                    if (p.z.p)
                        y[c][ip] = mul2(y[c][ip], mul2(z[c], make_float2(logistic<T>(z[c].x), logistic<T>(z[c].y))));
                }
                float2 o[kCh];
#pragma unroll
                for (int c = 0; c < kCh; ++c) o[c] = y[c][ip];
                put_lane_pair<T, kCh>(in, ip, o);
            }
            if (kVec && at.width == 32 * kCh) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tc::tma_store_4d(&maps.out[0], in, (int)at.c0, (int)t0, (int)at.b, 0);
                    tc::bulk_commit();
                }
            } else {
                __syncwarp();
                write_rows<T, kCh>(in, p.o, p, at, t0);
            }
        }
        __syncwarp();       // the stage and the rows have been read
        k ^= 1;
        round ^= k == 0;
        parity ^= 1;
    }
    if (kVec && kOut && lane == 0) tc::bulk_wait_all();
    float *last = kMode == kEnds ? sp.h : kOut && at.seg == sp.n - 1 ? p.hT : nullptr;
    if (last && w == (int)((at.ch1 - at.ch0 - 1) % W)) {    // what the last chunk handed on
        for (int q = 0; q < Q; ++q) {
            const float4 v = load4(to.slot + 512 * q);
            const float h[4] = {v.x, v.y, v.z, v.w};
            store_states<kCh>(last, kMode == kEnds ? at.row : at.b, p, at, q, h);
        }
    }
    if (kMode == kEnds) {
#pragma unroll
        for (int c = 0; c < kCh; ++c) sums[w][lane * kCh + c] = total[c].x + total[c].y;
        __syncthreads();
        for (int i = threadIdx.x; i < at.width; i += 32 * W) {
            float t = 0.f;
            for (int k2 = 0; k2 < W; ++k2) t += sums[k2][i];
            sp.sum[at.row * p.C + at.c0 + i] = t;
        }
    }
}

// Where the backward kernel leaves what is summed later, all float:
//   rows [tiles][B T][2][NP]: dB and dC of a tile's channels
//   chan [B][n][C][N + 2]: dA, then dD and ddt_bias, of a segment
struct Parts {
    float *rows, *chan;
};

// kEnd: no gradients but that of the state before the segment if nothing comes from behind it (Split).
template <typename T, int kCh, int kN, bool kEnd, bool kVec>
__global__ void __launch_bounds__(kCh == 2 ? 256 : 384, 1)
ssm_bwd_kernel(const __grid_constant__ SsmProblem p, const __grid_constant__ Maps maps, const Split sp,
               const float4 *marks, const Parts parts, unsigned int *err) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 chan[kCh == 2 ? 8 : 12][32 * kCh];
    constexpr int kSt = 4 / kCh, kIn = 4, kRow = kTok * 32 * kCh;
    using R = Ring<T, kCh>;
    const int W = blockDim.x / 32, N = kN ? kN : p.N, Q = R::steps(N), NP = R::padded(N);
    R ring(smem, W, N, true);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G, kCh);
    const Place<kCh> at(p, tl, sp, sp.n);
    if (!kEnd)
        for (int q = 0; q < Q; ++q) ring.sums[(w * Q + q) * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    ring.begin(p, at, W, N, kEnd ? nullptr : sp.n > 1 ? sp.g : p.dhT, sp.n > 1 ? at.row : at.b);
    float bias[kCh], D[kCh], dD[kCh], dbias[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        bias[c] = p.dt_bias ? p.dt_bias[at.channel(c)] : 0.f;
        D[c] = p.D ? p.D[at.channel(c)] : 0.f;
        dD[c] = dbias[c] = 0.f;
    }
    float2 *rows = ring.rows + w * 2 * kPairs * NP;
    float *turn = ring.turn + w * 32 * kTurn;
    const size_t stage_bytes = R::stage_bytes(kIn, N);
    auto stage = [&](int k) { return reinterpret_cast<T *>(ring.stage + (2 * w + k) * stage_bytes); };
    const int64_t chunks = (p.T + kTok - 1) / kTok, steps = at.ch1 - at.ch0;
    // the chunk into buffer k of the stage, by one lane where TMA does it
    auto fetch = [&](int64_t step, int k) {
        if (step >= steps) return;
        T *to = stage(k);
        const int64_t t0 = (at.ch1 - 1 - step) * kTok;
        if (kVec) {
            if (lane == 0) {
                uint64_t *bar = ring.full + 2 * w + k;
                tc::bulk_wait_read_all();       // the gradients that were there
                tc::mbar_arrive_expect_tx(bar, ((p.z.p ? 4 : 3) * kRow + 2 * kTok * N) * (int)sizeof(T));
                const int c = (int)at.c0, b = (int)at.b, t = (int)t0, n = (int)at.g * N;
                tc::tma_load_4d(to, &maps.in[0], bar, c, t, b, 0);
                tc::tma_load_4d(to + kRow, &maps.in[1], bar, c, t, b, 0);
                tc::tma_load_4d(to + 2 * kRow, &maps.in[3], bar, c, t, b, 0);
                if (p.z.p) tc::tma_load_4d(to + 3 * kRow, &maps.in[2], bar, c, t, b, 0);
                tc::tma_load_4d(to + kIn * kRow, &maps.b, bar, n, t, b, 0);
                tc::tma_load_4d(to + kIn * kRow + kTok * N, &maps.c, bar, n, t, b, 0);
            }
        } else {
            stage_rows<T>(at.template channels<T>(p.u), t0, p.T, to);
            stage_rows<T>(at.template channels<T>(p.dt), t0, p.T, to + kRow);
            stage_rows<T>(at.template channels<T>(p.go), t0, p.T, to + 2 * kRow);
            if (p.z.p) stage_rows<T>(at.template channels<T>(p.z), t0, p.T, to + 3 * kRow);
            stage_rows<T>(at.template rows<T>(p.Bm, N), t0, p.T, to + kIn * kRow);
            stage_rows<T>(at.template rows<T>(p.Cm, N), t0, p.T, to + kIn * kRow + kTok * N);
        }
    };
    const Link from = ring.link(w == 0 ? W - 1 : w - 1, Q), to = ring.link(w, Q);
    const uint32_t full = tc::smem_u32(ring.full + 2 * w);
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!try_wait(bar, parity)) dead = wait_on(bar, parity, dead, err);
    };
    int k = 0;
    uint32_t round = 0, parity = 0;     // of the stage's buffer, and of the hand-overs
    fetch(w, 0);
    for (int64_t step = w; step < steps; step += W) {
        const int64_t ch = at.ch1 - 1 - step, t0 = ch * kTok;
        const float4 *mark = marks + ((at.b * chunks + ch) * tl.all + at.tile) * Q * 32 + lane;
        float4 mk;                  // a step's states come while the one before is worked on
        if (!kEnd) mk = mark[0];
        if (kVec) wait(full + 8 * k, round);
        else __syncwarp();
        T *in = stage(k);
        widen_rows<T, kN>(in + kIn * kRow, rows, N);
        float2 d[kCh][kPairs], x[kCh][kPairs], dy[kCh][kPairs];
        float2 y[kCh][kPairs], gB[kCh][kPairs], wA[kCh][kPairs];
        step_sizes<T, kCh>(in + kRow, bias, p.softplus, p.T - t0, at.mine, d);
#pragma unroll
        for (int ip = 0; ip < kPairs; ++ip) {
            float2 u[kCh], go[kCh], z[kCh];
            lane_pair<T, kCh>(in, ip, u);
            lane_pair<T, kCh>(in + 2 * kRow, ip, go);
            if (p.z.p) lane_pair<T, kCh>(in + 3 * kRow, ip, z);
#pragma unroll
            for (int c = 0; c < kCh; ++c) {
                x[c][ip] = mul2(d[c][ip], u[c]);
                dy[c][ip] = go[c];
                if (p.z.p)
                    dy[c][ip] = mul2(go[c], mul2(z[c], make_float2(logistic<T>(z[c].x), logistic<T>(z[c].y))));
                if (c >= at.mine) x[c][ip] = dy[c][ip] = both(0.f);     // (TMA brings the next group's channels)
                y[c][ip] = gB[c][ip] = wA[c][ip] = both(0.f);
            }
        }
        __syncwarp();
        fetch(step + W, k ^ 1);
        // Sums across the lanes: a lane leaves its values in its row of turn; a step's are dC and dB of kSt states
        // of 8 tokens (2 tokens side by side), [2][kSt][kTok]. kCh = 2: two steps' values, 64 in all. Lane l
        // adds the columns 2 l and 2 l + 1 and has two tokens of dC or dB of one state.
#pragma unroll 1
        for (int q = 0; q < Q; ++q) {
            float2 A[4], a[4][kPairs], s[4][kPairs];
            float *mine = turn + lane * kTurn + (kCh == 2 ? q % 2 * 32 : 0);
            ring.load_a(q, A);
            if (kEnd) {
#pragma unroll
                for (int ip = 0; ip < kPairs; ++ip)
#pragma unroll
                    for (int j = 0; j < 4; ++j) a[j][ip] = decay2(A[j], d[j / kSt][ip]);
                wait(from.bar + 8 * q, parity);
                const float4 v = load4(from.slot + 512 * q);
                float G[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int ip = kPairs - 1; ip >= 0; --ip) {
                    float2 c[kSt];
                    load_bc<kSt>(rows + (kPairs + ip) * NP, q, c);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 g = mul2(c[j % kSt], dy[j / kSt][ip]);
                        G[j] = a[j][ip].y * (g.y + G[j]);
                        G[j] = a[j][ip].x * (g.x + G[j]);
                    }
                }
                store4(to.slot + 512 * q, G);
                hand_over(to.bar + 8 * q, lane);
                continue;
            }
            float h[4] = {mk.x, mk.y, mk.z, mk.w};
            if (q + 1 < Q) mk = mark[(q + 1) * 32];
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                float2 b[kSt], c[kSt], dC[kSt];
                load_bc<kSt>(rows + ip * NP, q, b);
                load_bc<kSt>(rows + (kPairs + ip) * NP, q, c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[j][ip] = decay2(A[j], d[j / kSt][ip]);
                    s[j][ip] = mul2(b[j % kSt], x[j / kSt][ip]);
                    // s: the states after the tokens
                    s[j][ip].x = fmaf(a[j][ip].x, ip ? s[j][ip ? ip - 1 : 0].y : h[j], s[j][ip].x);
                    s[j][ip].y = fmaf(a[j][ip].y, s[j][ip].x, s[j][ip].y);
                    y[j / kSt][ip] = fma2(c[j % kSt], s[j][ip], y[j / kSt][ip]);
                    dC[j % kSt] = j < kSt ? mul2(s[j][ip], dy[0][ip]) : fma2(s[j][ip], dy[j / kSt][ip], dC[j % kSt]);
                }
#pragma unroll
                for (int n = 0; n < kSt; ++n) *reinterpret_cast<float2 *>(mine + n * kTok + 2 * ip) = dC[n];
            }
            wait(from.bar + 8 * q, parity);
            const float4 v = load4(from.slot + 512 * q);
            float G[4] = {v.x, v.y, v.z, v.w};      // what comes from the tokens after
            // the walk, which the next warp waits for; a becomes the gradient of the state, the state before a
            // token becomes w (that before the first token: h)
#pragma unroll
            for (int ip = kPairs - 1; ip >= 0; --ip) {
                float2 c[kSt];
                load_bc<kSt>(rows + (kPairs + ip) * NP, q, c);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 g = mul2(c[j % kSt], dy[j / kSt][ip]);
                    g.y += G[j];
                    G[j] = a[j][ip].y * g.y;
                    s[j][ip].x *= G[j];
                    g.x += G[j];
                    G[j] = a[j][ip].x * g.x;
                    if (ip) s[j][ip - 1].y *= G[j];
                    else h[j] *= G[j];
                    a[j][ip] = g;
                }
            }
            store4(to.slot + 512 * q, G);
            hand_over(to.bar + 8 * q, lane);
            float2 dA[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dA[j] = both(0.f);
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                float2 b[kSt], dB[kSt];
                load_bc<kSt>(rows + ip * NP, q, b);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 g = a[j][ip], wt = make_float2(ip ? s[j][ip ? ip - 1 : 0].y : h[j], s[j][ip].x);
                    gB[j / kSt][ip] = fma2(g, b[j % kSt], gB[j / kSt][ip]);
                    wA[j / kSt][ip] = fma2(wt, A[j], wA[j / kSt][ip]);
                    dA[j] = fma2(wt, d[j / kSt][ip], dA[j]);
                    dB[j % kSt] = j < kSt ? mul2(g, x[0][ip]) : fma2(g, x[j / kSt][ip], dB[j % kSt]);
                }
#pragma unroll
                for (int n = 0; n < kSt; ++n) *reinterpret_cast<float2 *>(mine + (kSt + n) * kTok + 2 * ip) = dB[n];
            }
            // (a chunk's sum first: those of thousands of tokens go up in two steps)
            float4 *sum = ring.sums + (w * Q + q) * 32 + lane;
            const float4 all = *sum;
            *sum = make_float4(all.x + (dA[0].x + dA[0].y), all.y + (dA[1].x + dA[1].y), all.z + (dA[2].x + dA[2].y),
                               all.w + (dA[3].x + dA[3].y));
            if (kCh == 1 || q % 2 == 1 || q == Q - 1) {
                __syncwarp();
                float2 v = both(0.f);
#pragma unroll
                for (int l = 0; l < 32; ++l) v = add2(v, *reinterpret_cast<const float2 *>(turn + l * kTurn + 2 * lane));
                __syncwarp();
                const int at_q = kCh == 2 ? q / 2 * 2 + lane / 16 : q;              // the step,
                const int col = 2 * (kCh == 2 ? lane % 16 : lane);                  // [2][kSt][kTok]
                const int n = kSt * at_q + col / kTok % kSt, i = col % kTok, dB_ = col / (kSt * kTok);
                if (n < N && at_q <= q) {
                    float *out = parts.rows + (((at.tile * p.B + at.b) * p.T + t0 + i) * 2 + (1 - dB_)) * NP + n;
                    if (t0 + i < p.T) out[0] = v.x;
                    if (t0 + i + 1 < p.T) out[2 * NP] = v.y;
                }
            }
        }
        if (kEnd) {
            __syncwarp();       // the stage and the rows have been read
            k ^= 1;
            round ^= k == 0;
            parity ^= 1;
            continue;
        }
        float2 sD[kCh], sbias[kCh];
#pragma unroll
        for (int c = 0; c < kCh; ++c) sD[c] = sbias[c] = both(0.f);
#pragma unroll
        for (int ip = 0; ip < kPairs; ++ip) {
            float2 u[kCh], raw[kCh], go[kCh], z[kCh], du[kCh], ddt[kCh], dz[kCh];
            lane_pair<T, kCh>(in, ip, u);
            lane_pair<T, kCh>(in + kRow, ip, raw);
            lane_pair<T, kCh>(in + 2 * kRow, ip, go);
            if (p.z.p) lane_pair<T, kCh>(in + 3 * kRow, ip, z);
#pragma unroll
            for (int c = 0; c < kCh; ++c) {
                ddt[c] = fma2(wA[c][ip], both(kLn2), mul2(u[c], gB[c][ip]));
                if (p.softplus) {
                    const float2 r = add2(raw[c], both(bias[c]));
                    ddt[c] = mul2(ddt[c], make_float2(logistic<float>(r.x), logistic<float>(r.y)));
                }
                if (2 * ip >= p.T - t0) ddt[c].x = 0.f;         // tokens that do not exist
                if (2 * ip + 1 >= p.T - t0) ddt[c].y = 0.f;
                du[c] = fma2(both(D[c]), dy[c][ip], mul2(d[c][ip], gB[c][ip]));
                sbias[c] = add2(sbias[c], ddt[c]);
                sD[c] = fma2(dy[c][ip], u[c], sD[c]);
                if (p.z.p) {
                    const float2 yy = fma2(both(D[c]), u[c], y[c][ip]);
                    dz[c] = mul2(mul2(go[c], yy), make_float2(act_grad<T>(z[c].x, 1), act_grad<T>(z[c].y, 1)));
                }
            }
            put_lane_pair<T, kCh>(in, ip, du);
            put_lane_pair<T, kCh>(in + kRow, ip, ddt);
            if (p.dz) put_lane_pair<T, kCh>(in + 3 * kRow, ip, dz);
        }
#pragma unroll
        for (int c = 0; c < kCh; ++c) {
            dD[c] += sD[c].x + sD[c].y;
            dbias[c] += sbias[c].x + sbias[c].y;
        }
        if (kVec && at.width == 32 * kCh) {
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::tma_store_4d(&maps.out[0], in, (int)at.c0, (int)t0, (int)at.b, 0);
                tc::tma_store_4d(&maps.out[1], in + kRow, (int)at.c0, (int)t0, (int)at.b, 0);
                if (p.dz) tc::tma_store_4d(&maps.out[2], in + 3 * kRow, (int)at.c0, (int)t0, (int)at.b, 0);
                tc::bulk_commit();
            }
        } else {
            __syncwarp();
            write_rows<T, kCh>(in, p.du, p, at, t0);
            write_rows<T, kCh>(in + kRow, p.ddt, p, at, t0);
            if (p.dz) write_rows<T, kCh>(in + 3 * kRow, p.dz, p, at, t0);
        }
        __syncwarp();       // the stage and the rows have been read
        k ^= 1;
        round ^= k == 0;
        parity ^= 1;
    }
    if (kVec && lane == 0) tc::bulk_wait_all();
    float *first = kEnd ? sp.g : at.seg == 0 ? p.dh0 : nullptr;
    if (first && w == (int)((steps - 1) % W)) {             // what the first token handed on
        for (int q = 0; q < Q; ++q) {
            const float4 v = load4(to.slot + 512 * q);
            const float G[4] = {v.x, v.y, v.z, v.w};
            store_states<kCh>(first, kEnd ? at.row : at.b, p, at, q, G);
        }
    }
    if (kEnd) return;
#pragma unroll
    for (int c = 0; c < kCh; ++c) chan[w][lane * kCh + c] = make_float2(dD[c], dbias[c]);
    __syncthreads();
    // the warps' sums in order: a thread for each channel and state (state fastest)
    for (int k2 = threadIdx.x; k2 < at.width * (N + 2); k2 += blockDim.x) {
        const int ci = k2 / (N + 2), n = k2 % (N + 2), l = ci / kCh, j = ci % kCh * kSt + n % kSt;
        float s = 0.f;
        for (int i = 0; i < W; ++i) {
            if (n < N) s += reinterpret_cast<const float *>(ring.sums + (i * Q + n / kSt) * 32 + l)[j];
            else s += n == N ? chan[i][ci].x : chan[i][ci].y;
        }
        parts.chan[(at.row * p.C + at.c0 + ci) * (N + 2) + n] = s;
    }
}

// dB and dC from the tiles' parts, each added in order.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_rows_kernel(const __grid_constant__ SsmProblem p, const Parts parts, const Tiles tl) {
    const int NP = (p.N + 3) / 4 * 4;
    const int64_t rows = p.B * p.T, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t n = id % NP, k = id / NP % 2, g = id / (2 * NP) % p.G, row = id / (2 * NP) / p.G;
    if (row >= rows || n >= p.N) return;
    float s = 0.f;
    for (int i = 0; i < tl.per_group; ++i)
        s += parts.rows[(((g * tl.per_group + i) * rows + row) * 2 + k) * NP + n];
    put(static_cast<T *>(k ? p.dCm : p.dBm) + (row * p.G + g) * p.N + n, s);
}
// What the segments start from, from what they end with if they start from zero: in their order forward, or back.
__global__ void __launch_bounds__(256)
ssm_join_kernel(const __grid_constant__ SsmProblem p, const Split sp, int back) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, cn = p.C * p.N, b = id / cn, i = id - b * cn, c = i / p.N;
    if (b >= p.B) return;
    const float A = scale_a(p.A[i]), *from = back ? p.dhT : p.h0;
    float v = from ? from[id] : 0.f, *x = (back ? sp.g : sp.h) + b * sp.n * cn + i;
    const float *sum = sp.sum + b * sp.n * p.C + c;
#pragma unroll 4
    for (int k = 0; k < sp.n; ++k) {
        const int seg = back ? sp.n - 1 - k : k;
        const float end = x[seg * cn], a = exp2f(A * sum[seg * p.C]);
        x[seg * cn] = v;
        v = fmaf(a, v, end);
    }
}
// dA, dD and ddt_bias from the segments' parts.
__global__ void __launch_bounds__(256)
ssm_chan_kernel(const __grid_constant__ SsmProblem p, const Parts parts, int64_t rows) {
    const int64_t w = p.N + 2, id = (int64_t)blockIdx.x * 256 + threadIdx.x, c = id / w, n = id % w;
    if (c >= p.C) return;
    float s = 0.f;
#pragma unroll 4
    for (int64_t b = 0; b < rows; ++b) s += parts.chan[(b * p.C + c) * w + n];
    if (n < p.N) p.dA[c * p.N + n] = s;
    else if (n == p.N) { if (p.dD) p.dD[c] = s; }
    else if (p.dbias) p.dbias[c] = s;
}

struct Quad {                       // four states of a channel
    float2 a, b;
};
__device__ __forceinline__ Quad quad(float4 v) { return Quad{make_float2(v.x, v.y), make_float2(v.z, v.w)}; }
__device__ __forceinline__ float4 vec4(const Quad &q) { return make_float4(q.a.x, q.a.y, q.b.x, q.b.y); }
__device__ __forceinline__ Quad operator*(const Quad &x, float y) { return Quad{mul2(x.a, both(y)), mul2(x.b, both(y))}; }
__device__ __forceinline__ Quad fmaq(const Quad &x, const Quad &y, const Quad &z) {
    return Quad{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)};
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
            const Quad h = fmaq(Quad{decay2(A.a, both(d)), decay2(A.b, both(d))}, quad(load_quad(S, n0, p.N)), x);
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

template <typename T, int kCh>
int ring_warps(const SsmProblem &p, int in, bool backward, int most) {
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    int W = most;
    // (the backward kernel has 4 KB of its own)
    while (W > 1 && Ring<T, kCh>::bytes(W, in, p.N, backward) > 222 * 1024) W = W > 8 ? W - 4 : W / 2;
    return (int)std::min<int64_t>(W, chunks);
}

// A map of [B, T, cols] rows.
bool rows_map(CUtensorMap *m, const void *base, int io, int64_t cols, int64_t T, int64_t B, int64_t st, int64_t sb,
              int box_cols) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t es = io == 0 ? 2 : 4;
    const cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)T, (cuuint64_t)B, 1};
    const cuuint64_t strides[3] = {(cuuint64_t)st * es, (cuuint64_t)sb * es, (cuuint64_t)sb * es};
    const cuuint32_t box[4] = {(cuuint32_t)box_cols, kTok, 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(m, io == 0 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
              const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The maps of a call; false where a map cannot be made.
bool make_maps(const SsmProblem &p, int ch, Maps *m) {
    const SsmRows *in[4] = {&p.u, &p.dt, &p.z, &p.go};
    void *const out[3] = {p.du ? p.du : p.o, p.ddt, p.dz};
    for (int i = 0; i < 4; ++i)
        if (in[i]->p && !rows_map(&m->in[i], in[i]->p, p.io, p.C, p.T, p.B, in[i]->t, in[i]->b, 32 * ch)) return false;
    for (int i = 0; i < 3; ++i)
        if (out[i] && !rows_map(&m->out[i], out[i], p.io, p.C, p.T, p.B, p.C, p.T * p.C, 32 * ch)) return false;
    return rows_map(&m->b, p.Bm.p, p.io, p.G * p.N, p.T, p.B, p.Bm.t, p.Bm.b, p.N) &&
           rows_map(&m->c, p.Cm.p, p.io, p.G * p.N, p.T, p.B, p.Cm.t, p.Cm.b, p.N);
}

// Whether the rows of all inputs, and the first channels and groups of the tiles, are on 16 bytes.
bool vectors(const SsmProblem &p) {
    const int es = p.io == 0 ? 2 : 4;
    for (const SsmRows *r : {&p.u, &p.dt, &p.z, &p.go, &p.Bm, &p.Cm})
        if (r->p && (reinterpret_cast<uintptr_t>(r->p) % 16 || r->b * es % 16 || r->t * es % 16)) return false;
    // (strides and coordinates that a tensor map holds)
    for (const SsmRows *r : {&p.u, &p.dt, &p.z, &p.go, &p.Bm, &p.Cm})
        if (r->p && (r->b >= int64_t(1) << 38 || r->t >= int64_t(1) << 38)) return false;
    return p.C / p.G * es % 16 == 0 && p.N * es % 16 == 0 && p.T * p.C < int64_t(1) << 38;
}

// Channels of a lane in the backward pass: two, which share the loads of B and C and the sums across
// lanes, where the states of a step fit shared memory.
int bwd_channels(const SsmProblem &p) {
    const char *e = getenv("SSM_CH");
    if (e) return atoi(e);
    return p.N <= 64 ? 2 : 1; }

// Segments of a sequence for CTAs of 32 ch channels. Cutting it costs two thirds of a walk more (and the join), so it is
// done where the tiles leave almost half of the SMs idle; two CTAs to an SM then, of at least 8 chunks.
// Measured: SPLIT_NOTE
Split split_of(const SsmProblem &p, int ch, int splits, int num_sms) {
    const int64_t chunks = (p.T + kTok - 1) / kTok, ctas = p.B * tiles_of(p.C, p.G, ch).all;
    int64_t n = 1;
    if (splits > 0) n = std::min({(int64_t)splits, chunks, std::max<int64_t>(1, (int64_t(1) << 30) / ctas)});
    else if (9 * ctas <= 5 * num_sms) n = std::min<int64_t>(2 * num_sms / ctas, chunks / 8);
    Split sp{};
    sp.chunks = (chunks + std::max<int64_t>(n, 1) - 1) / std::max<int64_t>(n, 1);
    sp.n = (int)((chunks + sp.chunks - 1) / sp.chunks);
    return sp;
}
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
// The segments' states of one direction, and their step sizes.
size_t split_state_bytes(const SsmProblem &p, const Split &sp) {
    return sp.n > 1 ? round256((size_t)p.B * sp.n * p.C * p.N * 4) : 0;
}
size_t split_sum_bytes(const SsmProblem &p, const Split &sp) {
    return sp.n > 1 ? round256((size_t)p.B * sp.n * p.C * 4) : 0;
}

struct BwdWorkspace {
    size_t marks, rows, chan, all;
};
BwdWorkspace bwd_workspace(const SsmProblem &p, const Split &sp) {
    auto round = round256;
    const int ch = bwd_channels(p);
    const Tiles tl = tiles_of(p.C, p.G, ch);
    const size_t chunks = (size_t)((p.T + kTok - 1) / kTok), Q = (size_t)(p.N + 4 / ch - 1) / (4 / ch);
    BwdWorkspace w;
    w.marks = round((size_t)p.B * chunks * tl.all * Q * 32 * 16);
    w.rows = round((size_t)tl.all * p.B * p.T * 2 * ((p.N + 3) / 4 * 4) * 4);
    w.chan = round((size_t)p.B * sp.n * p.C * (p.N + 2) * 4);
    w.all = w.marks + w.rows + w.chan + 2 * split_state_bytes(p, sp) + split_sum_bytes(p, sp);
    return w;
}

template <typename T, int kCh, int kN, int kMode, bool kVec>
cudaError_t run_fwd(const SsmProblem &p, const Maps &maps, const Split &sp, int segs, int warps, float4 *marks,
                    unsigned int *err, cudaStream_t s) {
    constexpr int in = kMode == kOutputs ? 3 : 2;
    const int W = (int)std::min<int64_t>(ring_warps<T, kCh>(p, in, false, warps), sp.chunks);
    const size_t smem = Ring<T, kCh>::bytes(W, in, p.N, false);
    const auto kernel = ssm_fwd_kernel<T, kCh, kN, kMode, kVec>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(p.B * segs * tiles_of(p.C, p.G, kCh).all), 32 * W, smem, s>>>(p, maps, sp, segs, marks, err);
    return cudaGetLastError();
}
template <typename T, int kCh, int kMode>
cudaError_t fwd(const SsmProblem &p, const Maps *maps, const Split &sp, int segs, int num_sms, float4 *marks,
                unsigned int *err, cudaStream_t s) {
    // 16 warps to an SM: of one ring where there are no more rings than SMs
    const int warps = p.B * segs * tiles_of(p.C, p.G, kCh).all <= num_sms ? 16 : 8;
    cudaError_t e;
    if (!maps) e = run_fwd<T, kCh, 0, kMode, false>(p, Maps{}, sp, segs, warps, marks, err, s);
    else if (p.N == 16) e = run_fwd<T, kCh, 16, kMode, true>(p, *maps, sp, segs, warps, marks, err, s);
    else e = run_fwd<T, kCh, 0, kMode, true>(p, *maps, sp, segs, warps, marks, err, s);
    if (e == cudaSuccess) count_launches(1);
    return e;
}
cudaError_t join(const SsmProblem &p, const Split &sp, bool back, cudaStream_t s) {
    ssm_join_kernel<<<(unsigned)((p.B * p.C * p.N + 255) / 256), 256, 0, s>>>(p, sp, back);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T, int kCh, int kN, bool kEnd, bool kVec>
cudaError_t run_bwd(const SsmProblem &p, const Maps &maps, const Split &sp, const float4 *marks, const Parts &parts,
                    unsigned int *err, cudaStream_t s) {
    const int W = (int)std::min<int64_t>(ring_warps<T, kCh>(p, 4, true, kCh == 2 ? 8 : 12), sp.chunks);
    const size_t smem = Ring<T, kCh>::bytes(W, 4, p.N, true);
    const auto kernel = ssm_bwd_kernel<T, kCh, kN, kEnd, kVec>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(p.B * sp.n * tiles_of(p.C, p.G, kCh).all), 32 * W, smem, s>>>(p, maps, sp, marks, parts, err);
    return cudaGetLastError();
}
template <typename T, int kCh, bool kEnd>
cudaError_t back(const SsmProblem &p, const Maps *maps, const Split &sp, const float4 *marks, const Parts &parts,
                 unsigned int *err, cudaStream_t s) {
    cudaError_t e;
    if (!maps) e = run_bwd<T, kCh, 0, kEnd, false>(p, Maps{}, sp, marks, parts, err, s);
    else if (p.N == 16) e = run_bwd<T, kCh, 16, kEnd, true>(p, *maps, sp, marks, parts, err, s);
    else e = run_bwd<T, kCh, 0, kEnd, true>(p, *maps, sp, marks, parts, err, s);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

template <typename T>
cudaError_t whole_fwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *err, cudaStream_t s) {
    Maps store;
    const bool vec = vectors(p);
    if (vec && !make_maps(p, 1, &store)) return cudaErrorInvalidResourceHandle;
    const Maps *maps = vec ? &store : nullptr;
    Split sp = split_of(p, 1, splits, num_sms);
    cudaError_t e = cudaSuccess;
    if (sp.n > 1) {
        sp.h = static_cast<float *>(ws);
        sp.sum = reinterpret_cast<float *>(static_cast<char *>(ws) + split_state_bytes(p, sp));
        e = fwd<T, 1, kEnds>(p, maps, sp, sp.n - 1, num_sms, nullptr, err, s);      // (nothing starts from the last one's end)
        if (e == cudaSuccess) e = join(p, sp, false, s);
    }
    return e == cudaSuccess ? fwd<T, 1, kOutputs>(p, maps, sp, sp.n, num_sms, nullptr, err, s) : e;
}
template <typename T, int kCh>
cudaError_t whole_bwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *err, cudaStream_t s) {
    Maps store;
    const bool vec = vectors(p);
    if (vec && !make_maps(p, kCh, &store)) return cudaErrorInvalidResourceHandle;
    const Maps *maps = vec ? &store : nullptr;
    Split sp = split_of(p, kCh, splits, num_sms);
    const BwdWorkspace lay = bwd_workspace(p, sp);
    char *at = static_cast<char *>(ws);
    float4 *marks = reinterpret_cast<float4 *>(at);
    const Parts parts{reinterpret_cast<float *>(at + lay.marks), reinterpret_cast<float *>(at + lay.marks + lay.rows)};
    cudaError_t e = cudaSuccess;
    if (sp.n > 1) {
        at += lay.marks + lay.rows + lay.chan;
        sp.h = reinterpret_cast<float *>(at);
        sp.g = reinterpret_cast<float *>(at + split_state_bytes(p, sp));
        sp.sum = reinterpret_cast<float *>(at + 2 * split_state_bytes(p, sp));
        e = fwd<T, kCh, kEnds>(p, maps, sp, sp.n, num_sms, nullptr, err, s);
        if (e == cudaSuccess) e = back<T, kCh, true>(p, maps, sp, nullptr, parts, err, s);
        if (e == cudaSuccess) e = join(p, sp, false, s);
        if (e == cudaSuccess) e = join(p, sp, true, s);
    }
    if (e == cudaSuccess) e = fwd<T, kCh, kMarks>(p, maps, sp, sp.n, num_sms, marks, err, s);
    if (e == cudaSuccess) e = back<T, kCh, false>(p, maps, sp, marks, parts, err, s);
    if (e != cudaSuccess) return e;
    const int64_t rows = p.B * p.T * p.G * 2 * ((p.N + 3) / 4 * 4), chan = p.C * (p.N + 2);
    ssm_rows_kernel<T><<<(unsigned)((rows + 255) / 256), 256, 0, s>>>(p, parts, tiles_of(p.C, p.G, kCh));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ssm_chan_kernel<<<(unsigned)((chan + 255) / 256), 256, 0, s>>>(p, parts, p.B * sp.n);
    if ((e = cudaGetLastError()) == cudaSuccess) count_launches(2);
    return e;
}

}  // namespace

size_t ssm_fwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms) {
    const Split sp = split_of(p, 1, splits, num_sms);
    return split_state_bytes(p, sp) + split_sum_bytes(p, sp);
}
size_t ssm_bwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms) {
    return bwd_workspace(p, split_of(p, bwd_channels(p), splits, num_sms)).all;
}

cudaError_t launch_ssm_fwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err, cudaStream_t s) {
    return p.io == 0 ? whole_fwd<__nv_bfloat16>(p, splits, num_sms, ws, dev_err, s)
                     : whole_fwd<float>(p, splits, num_sms, ws, dev_err, s);
}

cudaError_t launch_ssm_bwd(const SsmProblem &p, int splits, int num_sms, void *ws, unsigned int *dev_err, cudaStream_t s) {
    if (bwd_channels(p) == 2)
        return p.io == 0 ? whole_bwd<__nv_bfloat16, 2>(p, splits, num_sms, ws, dev_err, s)
                         : whole_bwd<float, 2>(p, splits, num_sms, ws, dev_err, s);
    return p.io == 0 ? whole_bwd<__nv_bfloat16, 1>(p, splits, num_sms, ws, dev_err, s)
                     : whole_bwd<float, 1>(p, splits, num_sms, ws, dev_err, s);
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
