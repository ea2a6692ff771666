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
// Forward, pairs of packed arithmetic are two states of a token. What a warp does between the state's arrival
// and its hand-over is all that is serial, and so it is 16 instructions for 4 states of 8 tokens; each token's d and d u are
// needed twice side by side, which costs the moves that the walk saves (16384 tokens of 4096 channels, bf16, 16 states,
// inputs and outputs 539 MB: 411 us; when it was built 423, and 448 with pairs of tokens). Backward, where registers are few, pairs are two
// tokens of a state: step sizes, inputs, B, C and sums are pairs as they come, and only the walk is scalar.
//
// Bound: 16 exponentials of a token of 32 channels take 64 cycles of a scheduler's share of the special function
// units, the four multiply-adds of each state 64 of its FP32 pipe; in the backward pass thirteen of them 208. Forward, on
// all 608 schedulers at 2.07 GHz, that is 107 us of the 411. What bounds it is the shared-memory data pipe: on its SM a
// chunk comes every 415 cycles, in 337 of which (82 %) that pipe moves a wavefront, most of them the reads of B, C, d u
// and d in each of the four steps. Gradients (4 x 2047 tokens of 2048 channels) have 87 us of multiply-adds and take 437, 345 of
// them in the backward kernel, whose two warps to a scheduler (255 registers) issue half of the time.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "gla_internal.h"
#include "launch.h"
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
// e takes its error from 2^x (2^-22) and from the rounding of x log2 e, which is |x| 2^-24 of the value (6e-7 of the step at
// x = -7, 1e-6 at -12, 4e-6 at -60). fp32 calls put back what the rounding left out, to first order: their steps are good to
// 8 2^-24 whatever x is (16384 tokens of 4096 channels 464 us, 458 without). bf16 calls, whose dt has 2^-9 |x| of the step to itself, do not pay for that.
template <typename T>
__device__ __forceinline__ float softplus(float x) {
    const float a = fabsf(x), t = a * -kLog2e;
    float e = ex2(t);
    if (sizeof(T) == 4) {       // e^(-a - t ln 2); where t is not finite that is infinite or NaN, and e is 0
        constexpr float kLn2Low = 0.6931471805599453 - (double)kLn2;
        e = fmaf(e, fminf(fmaf(t, -kLn2Low, -fmaf(t, kLn2, a)), 1.f), e);
    }
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
template <typename T>
__device__ __forceinline__ float step_size(float x, int on) { return on ? softplus<T>(x) : x; }

// Tensor maps of the rows: boxes of kTok tokens by a tile's channels (or a group's states).
struct Maps {
    CUtensorMap in[4], b, c, out[3];
};

// B and C of the chunk as floats, the values of two tokens side by side as the packed arithmetic takes
// them: from[2][kTok][row] -> to[2][kTok / 2][NP] float2, NP = N up to a multiple of 4, zero past N.
template <typename T, int kN>
__device__ __forceinline__ void widen_rows(const T *from, float2 *to, int N, int row) {
    const int lane = threadIdx.x % 32, NP = (N + 3) / 4 * 4;
    if constexpr (kN > 0) {     // four states at a time
#pragma unroll
        for (int k = lane; k < kTok * kN / 4; k += 32) {
            const int i = k / (kN / 4), q = k % (kN / 4);       // i: a pair of tokens of B, or of C
            float x[4], y[4];
            Pack<T, 4>::unpack(*reinterpret_cast<const typename Pack<T, 4>::raw *>(from + 2 * i * kN + 4 * q), x);
            Pack<T, 4>::unpack(*reinterpret_cast<const typename Pack<T, 4>::raw *>(from + (2 * i + 1) * kN + 4 * q), y);
            float4 *t = reinterpret_cast<float4 *>(to + i * NP + 4 * q);
            t[0] = make_float4(x[0], y[0], x[1], y[1]);
            t[1] = make_float4(x[2], y[2], x[3], y[3]);
        }
    } else {
        for (int n = lane; n < NP; n += 32)
#pragma unroll
            for (int i = 0; i < kTok; ++i)      // (pairs of tokens of B, then of C)
                to[i * NP + n] = n < N ? make_float2(get(from + 2 * i * row + n), get(from + (2 * i + 1) * row + n)) : both(0.f);
    }
}

// The same for the forward walk, as they are: from[2][kTok][row] -> to[2][kTok][NP] floats.
template <typename T, int kN>
__device__ __forceinline__ void widen_tokens(const T *from, float *to, int N, int row) {
    const int lane = threadIdx.x % 32, NP = (N + 3) / 4 * 4;
    if (kN > 0 || row == NP) {          // (what is past N in a row is zero)
#pragma unroll
        for (int k = lane; k < 2 * kTok * (kN > 0 ? kN : NP) / 4; k += 32) {
            float x[4];
            Pack<T, 4>::unpack(*reinterpret_cast<const typename Pack<T, 4>::raw *>(from + 4 * k), x);
            *reinterpret_cast<float4 *>(to + 4 * k) = make_float4(x[0], x[1], x[2], x[3]);
        }
    } else {
        for (int n = lane; n < NP; n += 32)
#pragma unroll
            for (int i = 0; i < 2 * kTok; ++i) to[i * NP + n] = n < N ? get(from + i * row + n) : 0.f;
    }
}

// Hand-overs. Addresses are those of shared memory, so that a step's are immediate offsets of a chunk's.
struct Link {
    uint32_t bar, slot;             // step 0 of a warp (32 slots of 16 bytes and one barrier to a step)
};
__device__ __forceinline__ float4 load4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store4(uint32_t at, const float (&v)[4]) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                 : "memory");
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
// gives up lets what it has asked for land (bounded, too, as the shared memory of a CTA that ends is another's): the
// chunk in buffer k of its stage, and the next one. From then on it asks for nothing, waits for nothing and goes on
// with what is there.
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, bool dead, uint64_t *full, int k, uint32_t round,
                                        unsigned int *err) {
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
    tc::mbar_wait(full + k, round);
    tc::mbar_wait(full + (k ^ 1), round ^ k);
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

// Where a CTA is: a sequence (a segment of it), a group of channels and 32 kCh of them. (All of it fits 32 bits, which saves
// registers: 16384 tokens of 4096 channels 418 -> 411 us, gradients of 4 x 2047 tokens of 2048 channels 438 -> 426.)
template <int kCh>
struct Place {
    int b, row, tile, g, c0;        // row: b n + the segment; c0: the first channel
    int in;                         // where it is in the inputs
    int seg;
    int ch0, ch1;                   // chunks
    int width, mine;                // channels of the tile, of the lane
    __device__ Place(const SsmProblem &p, const Tiles &tl, const Split &sp, int segs) {
        const int all = (int)tl.all, i = (int)(blockIdx.x / all), cg = (int)(p.C / p.G);
        tile = (int)(blockIdx.x % all);
        b = i / segs;
        seg = i - b * segs;
        row = b * sp.n + seg;
        ch0 = seg * (int)sp.chunks;
        ch1 = min(ch0 + (int)sp.chunks, (int)((p.T + kTok - 1) / kTok));
        g = tile / tl.per_group;
        const int first = (tile - g * tl.per_group) * 32 * kCh;
        width = min(32 * kCh, cg - first);
        c0 = g * cg + first;
        in = g * (int)p.group + first;
        mine = max(0, min(kCh, width - kCh * (int)(threadIdx.x % 32)));
    }
    // Channel j of the lane; the tile's first one where there is none.
    __device__ int channel(int j) const { return c0 + (j < mine ? threadIdx.x % 32 * kCh + j : 0); }
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
//   slot[W][Q][32] float4: what a warp hands on, [kCh][kSt];  A[Q][32] float4: A log2 e (backward [Q][2][32]: twice each)
//   sums[W][Q][32] float4 (backward): dA;  turn[W][32][kTurn] float (backward): sums across lanes
//   rows[W][2][kPairs][NP] float2: B and C of a warp's chunk (forward [W][2][kTok][NP] float);  bar[W][Q]
//   stage[W][2]: a chunk as it lies in memory, on its way while the one before it is worked on:
//     kIn tensors [kTok][32 kCh], then B and C [kTok][row];  full[W][2]: it is there
//   dx[W][kPairs][kCh][32] float4 (forward): d u and d of a warp's chunk
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
    static __host__ __device__ size_t stage_bytes(int in, int row) {
        return ((size_t)in * kTok * 32 * kCh * sizeof(T) + 2 * kTok * (size_t)row * sizeof(T) + 127) / 128 * 128;
    }
    static __host__ __device__ size_t round(size_t n) { return (n + 127) / 128 * 128; }
    static __host__ __device__ size_t stage_at(int W, int N, bool backward) {
        const size_t Q = steps(N);
        return W * Q * 32 * 16 * (backward ? 2 : 1) + Q * (backward ? 2 : 1) * 32 * 16 + (backward ? round(W * 32 * kTurn * 4) : 0) +
               round((size_t)W * 2 * kPairs * padded(N) * 8) + round(W * (Q + 2) * 8);
    }
    static __host__ __device__ size_t bytes(int W, int in, int N, int row, bool backward) {
        return stage_at(W, N, backward) + 2 * W * stage_bytes(in, row) + (backward ? 0 : W * kPairs * kCh * 32 * 16);
    }
    __device__ Ring(unsigned char *smem, int W, int N, bool backward) {
        const int Q = steps(N);
        slot = reinterpret_cast<float4 *>(smem);
        A = slot + W * Q * 32;
        sums = A + Q * (backward ? 2 : 1) * 32;
        turn = reinterpret_cast<float *>(sums + (backward ? W * Q * 32 : 0));
        unsigned char *after = reinterpret_cast<unsigned char *>(turn) + (backward ? round(W * 32 * kTurn * 4) : 0);
        rows = reinterpret_cast<float2 *>(after);
        bar = reinterpret_cast<uint64_t *>(after + round((size_t)W * 2 * kPairs * padded(N) * 8));
        full = bar + W * Q;
        stage = smem + stage_at(W, N, backward);
    }
    // A, the barriers, and the states that the first chunk takes over, as if from the last warp; the CTA synchronises.
    template <bool kBack>
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
            if (kBack) {
                A[2 * q * 32 + lane] = make_float4(a[0], a[0], a[1], a[1]);
                A[(2 * q + 1) * 32 + lane] = make_float4(a[2], a[2], a[3], a[3]);
            } else {
                A[q * 32 + lane] = make_float4(a[0], a[1], a[2], a[3]);
            }
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
            for (int ip = 0; ip < kPairs; ++ip) d[c][ip] = make_float2(softplus<T>(d[c][ip].x), softplus<T>(d[c][ip].y));
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

// The step's states of a token's row of B (or C), in pairs.
template <int kSt>
__device__ __forceinline__ void load_states_row(const float *row, int q, float2 (&v)[2]) {
    if constexpr (kSt == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(row + 4 * q);
        v[0] = make_float2(x.x, x.y);
        v[1] = make_float2(x.z, x.w);
    } else {
        v[0] = v[1] = *reinterpret_cast<const float2 *>(row + 2 * q);
    }
}

// What a forward walk leaves: outputs and the last state; the states before each chunk (marks
// [B][chunks][tiles][Q][32] float4), which the backward walk needs; a segment's last state and step sizes (Split).
enum { kOutputs = 0, kMarks = 1, kEnds = 2 };

// kN: N, if known at compile time. segs: segments of a sequence that this call walks over.
template <typename T, int kCh, int kN, int kMode>
__global__ void __launch_bounds__(512, 1)
ssm_fwd_kernel(const __grid_constant__ SsmProblem p, const __grid_constant__ Maps maps, const Split sp, int segs,
               float4 *marks, unsigned int *err) {
    tc::pdl_launch_dependents();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float sums[kMode == kEnds ? 16 : 1][32 * kCh];
    constexpr bool kOut = kMode == kOutputs;
    constexpr int kSt = 4 / kCh, kIn = kOut ? 3 : 2, kRow = kTok * 32 * kCh;
    using R = Ring<T, kCh>;
    const int W = blockDim.x / 32, N = kN ? kN : p.N, row = kN ? kN : p.row, Q = R::steps(N), NP = R::padded(N);
    R ring(smem, W, N, false);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G, kCh);
    const Place<kCh> at(p, tl, sp, segs);
    tc::pdl_wait_prerequisites();
    ring.template begin<false>(p, at, W, N, kMode == kEnds ? nullptr : sp.n > 1 ? sp.h : p.h0, sp.n > 1 ? at.row : at.b);
    float bias[kCh], D[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        bias[c] = p.dt_bias ? p.dt_bias[at.channel(c)] : 0.f;
        D[c] = p.D ? p.D[at.channel(c)] : 0.f;
    }
    float *rows = reinterpret_cast<float *>(ring.rows) + w * 2 * kTok * NP;
    const size_t stage_bytes = R::stage_bytes(kIn, row);
    auto stage = [&](int k) { return reinterpret_cast<T *>(ring.stage + (2 * w + k) * stage_bytes); };
    // d u of a chunk, and with outputs d: in registers d costs moves, as 128 are few (walks of no outputs have some left:
    // the marks of 4 x 2047 tokens of 2048 channels 92 us, 83 with d in registers; outputs of 16384 x 4096 411, 549 when they were)
    using DX = std::conditional_t<kOut, float4, float2>;
    DX *dx = reinterpret_cast<DX *>(ring.stage + 2 * W * stage_bytes) + w * kPairs * kCh * 32 + lane;
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    bool dead = false;                  // the warp has given up
    // the chunk into buffer k of the stage
    auto fetch = [&](int64_t ch, int k) {
        if (ch >= at.ch1 || dead) return;
        T *to = stage(k);
        const int64_t t0 = ch * kTok;
        if (lane == 0) {
            uint64_t *bar = ring.full + 2 * w + k;
            const bool z = kOut && p.z.p;
            tc::bulk_wait_read_all();       // the outputs that were there
            tc::mbar_arrive_expect_tx(bar, ((z ? 3 : 2) * kRow + 2 * kTok * row) * (int)sizeof(T));
            const int c = at.in, b = (int)at.b, t = (int)t0, n = (int)at.g * row;
            tc::tma_load_4d(to, &maps.in[0], bar, c, t, b, 0);
            tc::tma_load_4d(to + kRow, &maps.in[1], bar, c, t, b, 0);
            if (z) tc::tma_load_4d(to + 2 * kRow, &maps.in[2], bar, c, t, b, 0);
            tc::tma_load_4d(to + kIn * kRow, &maps.b, bar, n, t, b, 0);
            tc::tma_load_4d(to + kIn * kRow + kTok * row, &maps.c, bar, n, t, b, 0);
        }
    };
    const Link from = ring.link(w == 0 ? W - 1 : w - 1, Q), to = ring.link(w, Q);
    const uint32_t full = tc::smem_u32(ring.full + 2 * w);
    int k = 0;
    uint32_t round = 0, parity = 0;     // of the stage's buffer, and of the hand-overs
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!try_wait(bar, parity) && wait_on(bar, parity, dead, ring.full + 2 * w, k, round, err)) dead = true;
    };
    float2 total[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) total[c] = both(0.f);
    if (w != p.stall) fetch(at.ch0 + w, 0);
    for (int64_t ch = at.ch0 + w; ch < at.ch1; ch += W) {
        const int64_t t0 = ch * kTok;
        wait(full + 8 * k, round);
        T *in = stage(k);
        widen_tokens<T, kN>(in + kIn * kRow, rows, N, row);
        float2 d[kCh][kPairs], y[kCh][kTok];        // y: of even and odd states
        step_sizes<T, kCh>(in + kRow, bias, p.softplus, p.T - t0, at.mine, d);
#pragma unroll
        for (int ip = 0; ip < kPairs; ++ip) {
            float2 u[kCh];
            lane_pair<T, kCh>(in, ip, u);
#pragma unroll
            for (int c = 0; c < kCh; ++c) {
                const float2 x = c < at.mine ? mul2(d[c][ip], u[c]) : both(0.f);
                DX *at_dx = dx + (ip * kCh + c) * 32;
                if constexpr (kOut) *at_dx = make_float4(x.x, x.y, d[c][ip].x, d[c][ip].y);
                else *at_dx = x;
                y[c][2 * ip] = y[c][2 * ip + 1] = both(0.f);
                if (kMode == kEnds) total[c] = add2(total[c], d[c][ip]);
            }
        }
        __syncwarp();
        fetch(ch + W, k ^ 1);
#pragma unroll 1
        for (int q = 0; q < Q; ++q) {
            // pairs of states: (0, 1), (2, 3) of [kCh][kSt]
            const float4 av = ring.A[q * 32 + lane];
            const float2 A[2] = {make_float2(av.x, av.y), make_float2(av.z, av.w)};
            float2 a[kTok][2], s[kTok][2];
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                DX v[kCh];
                float2 of_d[kCh];
#pragma unroll
                for (int c = 0; c < kCh; ++c) {
                    v[c] = dx[(ip * kCh + c) * 32];
                    if constexpr (kOut) of_d[c] = make_float2(v[c].z, v[c].w);
                    else of_d[c] = d[c][ip];
                }
#pragma unroll
                for (int i = 2 * ip; i < 2 * ip + 2; ++i) {
                    float2 b[2];
                    load_states_row<kSt>(rows + i * NP, q, b);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = kCh == 1 ? 0 : j;
                        a[i][j] = decay2(A[j], both(i % 2 ? of_d[c].y : of_d[c].x));
                        s[i][j] = mul2(b[j], both(i % 2 ? v[c].y : v[c].x));
                    }
                }
            }
            wait(from.bar + 8 * q, parity);
            const float4 v = load4(from.slot + 512 * q);
            float2 h[2] = {make_float2(v.x, v.y), make_float2(v.z, v.w)};
            if (kMode == kMarks)
                marks[(((at.b * chunks + ch) * tl.all + at.tile) * Q + q) * 32 + lane] = v;
            // the walk, which the next warp waits for
#pragma unroll
            for (int i = 0; i < kTok; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) h[j] = s[i][j] = fma2(a[i][j], h[j], s[i][j]);
            const float last[4] = {h[0].x, h[0].y, h[1].x, h[1].y};
            store4(to.slot + 512 * q, last);
            hand_over(to.bar + 8 * q, lane);
            if (kOut) {
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    float2 c[2];
                    load_states_row<kSt>(rows + (kTok + i) * NP, q, c);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float2 &to_y = y[kCh == 1 ? 0 : j][i];
                        to_y = fma2(c[j], s[i][j], to_y);
                    }
                }
            }
        }
        if (kOut) {
            // outputs take the place of u in the stage, then leave in whole rows
#pragma unroll
            for (int ip = 0; ip < kPairs; ++ip) {
                float2 u[kCh], z[kCh], o[kCh];
                if (p.D) lane_pair<T, kCh>(in, ip, u);
                if (p.z.p) lane_pair<T, kCh>(in + 2 * kRow, ip, z);
#pragma unroll
                for (int c = 0; c < kCh; ++c) {
                    const float2 even = y[c][2 * ip], odd = y[c][2 * ip + 1];
                    o[c] = make_float2(even.x + even.y, odd.x + odd.y);
                    if (p.D) o[c] = fma2(both(D[c]), u[c], o[c]);
                    if (p.z.p) o[c] = mul2(o[c], mul2(z[c], make_float2(logistic<T>(z[c].x), logistic<T>(z[c].y))));
                }
                put_lane_pair<T, kCh>(in, ip, o);
            }
            tc::fence_proxy_async_smem();       // (TMA reads the outputs, and writes the next chunk over them)
            __syncwarp();
            if (p.tma_out && at.width == 32 * kCh) {
                if (lane == 0) {
                    tc::tma_store_4d(&maps.out[0], in, (int)at.c0, (int)t0, (int)at.b, 0);
                    tc::bulk_commit();
                }
            } else {
                write_rows<T, kCh>(in, p.o, p, at, t0);
            }
        }
        __syncwarp();       // the stage and the rows have been read
        k ^= 1;
        round ^= k == 0;
        parity ^= 1;
    }
    if (kOut && lane == 0) tc::bulk_wait_all();
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
template <typename T, int kCh, int kN, bool kEnd>
__global__ void __launch_bounds__(kCh == 2 ? 256 : 384, 1)
ssm_bwd_kernel(const __grid_constant__ SsmProblem p, const __grid_constant__ Maps maps, const Split sp,
               const float4 *marks, const Parts parts, unsigned int *err) {
    tc::pdl_launch_dependents();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 chan[kCh == 2 ? 8 : 12][32 * kCh];
    constexpr int kSt = 4 / kCh, kIn = 4, kRow = kTok * 32 * kCh;
    using R = Ring<T, kCh>;
    const int W = blockDim.x / 32, N = kN ? kN : p.N, row = kN ? kN : p.row, Q = R::steps(N), NP = R::padded(N);
    R ring(smem, W, N, true);
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32;
    const Tiles tl = tiles_of(p.C, p.G, kCh);
    const Place<kCh> at(p, tl, sp, sp.n);
    if (!kEnd)
        for (int q = 0; q < Q; ++q) ring.sums[(w * Q + q) * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    tc::pdl_wait_prerequisites();
    ring.template begin<true>(p, at, W, N, kEnd ? nullptr : sp.n > 1 ? sp.g : p.dhT, sp.n > 1 ? at.row : at.b);
    float bias[kCh], D[kCh], dD[kCh], dbias[kCh];
#pragma unroll
    for (int c = 0; c < kCh; ++c) {
        bias[c] = p.dt_bias ? p.dt_bias[at.channel(c)] : 0.f;
        D[c] = p.D ? p.D[at.channel(c)] : 0.f;
        dD[c] = dbias[c] = 0.f;
    }
    float2 *rows = ring.rows + w * 2 * kPairs * NP;
    float *turn = ring.turn + w * 32 * kTurn;
    const size_t stage_bytes = R::stage_bytes(kIn, row);
    auto stage = [&](int k) { return reinterpret_cast<T *>(ring.stage + (2 * w + k) * stage_bytes); };
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    const int last = at.ch1 - 1, steps = at.ch1 - at.ch0;
    bool dead = false;                  // the warp has given up
    // the chunk into buffer k of the stage
    auto fetch = [&](int step, int k) {
        if (step >= steps || dead) return;
        T *to = stage(k);
        const int t0 = (last - step) * kTok;
        if (lane == 0) {
            uint64_t *bar = ring.full + 2 * w + k;
            tc::bulk_wait_read_all();       // the gradients that were there
            tc::mbar_arrive_expect_tx(bar, ((p.z.p ? 4 : 3) * kRow + 2 * kTok * row) * (int)sizeof(T));
            const int c = at.in, b = (int)at.b, t = (int)t0, n = (int)at.g * row;
            tc::tma_load_4d(to, &maps.in[0], bar, c, t, b, 0);
            tc::tma_load_4d(to + kRow, &maps.in[1], bar, c, t, b, 0);
            tc::tma_load_4d(to + 2 * kRow, &maps.in[3], bar, c, t, b, 0);
            if (p.z.p) tc::tma_load_4d(to + 3 * kRow, &maps.in[2], bar, c, t, b, 0);
            tc::tma_load_4d(to + kIn * kRow, &maps.b, bar, n, t, b, 0);
            tc::tma_load_4d(to + kIn * kRow + kTok * row, &maps.c, bar, n, t, b, 0);
        }
    };
    const Link from = ring.link(w == 0 ? W - 1 : w - 1, Q), to = ring.link(w, Q);
    const uint32_t full = tc::smem_u32(ring.full + 2 * w);
    int k = 0;
    uint32_t round = 0, parity = 0;     // of the stage's buffer, and of the hand-overs
    auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!try_wait(bar, parity) && wait_on(bar, parity, dead, ring.full + 2 * w, k, round, err)) dead = true;
    };
    if (w != p.stall) fetch(w, 0);
    for (int step = w; step < steps; step += W) {
        const int ch = last - step, t0 = ch * kTok, left = (int)p.T - t0;
        const float4 *mark = marks + ((at.b * chunks + ch) * tl.all + at.tile) * Q * 32 + lane;
        float4 mk;                  // a step's states come while the one before is worked on
        if (!kEnd) mk = mark[0];
        wait(full + 8 * k, round);
        T *in = stage(k);
        widen_rows<T, kN>(in + kIn * kRow, rows, N, row);
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
            if constexpr (kEnd) {
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
            } else {
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
                // (tokens that do not exist have no part in dA: a last state that is not finite times their d of 0 is NaN)
                if (left < kTok) {
#pragma unroll
                    for (int i = 1; i < kTok; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (i >= left) (i % 2 ? s[j][i / 2].x : s[j][i / 2 - 1].y) = 0.f;
                }
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
                    for (int l = 0; l < 32; ++l)
                        v = add2(v, *reinterpret_cast<const float2 *>(turn + l * kTurn + 2 * lane));
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
        }
        if constexpr (!kEnd) {
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
            tc::fence_proxy_async_smem();           // (TMA reads the gradients, and writes the next chunk over them)
            __syncwarp();
            if (p.tma_out && at.width == 32 * kCh) {
                if (lane == 0) {
                    tc::tma_store_4d(&maps.out[0], in, (int)at.c0, (int)t0, (int)at.b, 0);
                    tc::tma_store_4d(&maps.out[1], in + kRow, (int)at.c0, (int)t0, (int)at.b, 0);
                    if (p.dz) tc::tma_store_4d(&maps.out[2], in + 3 * kRow, (int)at.c0, (int)t0, (int)at.b, 0);
                    tc::bulk_commit();
                }
            } else {
                write_rows<T, kCh>(in, p.du, p, at, t0);
                write_rows<T, kCh>(in + kRow, p.ddt, p, at, t0);
                if (p.dz) write_rows<T, kCh>(in + 3 * kRow, p.dz, p, at, t0);
            }
        }
        __syncwarp();       // the stage and the rows have been read
        k ^= 1;
        round ^= k == 0;
        parity ^= 1;
    }
    if (lane == 0) tc::bulk_wait_all();
    float *first = kEnd ? sp.g : at.seg == 0 ? p.dh0 : nullptr;
    if (first && w == (int)((steps - 1) % W)) {             // what the first token handed on
        for (int q = 0; q < Q; ++q) {
            const float4 v = load4(to.slot + 512 * q);
            const float G[4] = {v.x, v.y, v.z, v.w};
            store_states<kCh>(first, kEnd ? at.row : at.b, p, at, q, G);
        }
    }
    if constexpr (!kEnd) {
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
}

// What the segments start from, from what they end with if they start from zero: in their order forward, or back
// (blockIdx.y).
__global__ void __launch_bounds__(256)
ssm_join_kernel(const __grid_constant__ SsmProblem p, const Split sp) {
    constexpr int kAhead = 8;       // segments whose values are on their way together
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    const bool back = blockIdx.y == 1;
    const int cn = (int)(p.C * p.N), i = (int)(blockIdx.x * 256 + threadIdx.x);
    const int64_t b = blockIdx.z;
    if (i >= cn) return;
    const float A = scale_a(p.A[i]), *from = back ? p.dhT : p.h0;
    float v = from ? from[b * cn + i] : 0.f, *x = (back ? sp.g : sp.h) + b * sp.n * cn + i;
    const float *sum = sp.sum + b * sp.n * p.C + i / p.N;
    for (int k = 0; k < sp.n; k += kAhead) {
        float end[kAhead], a[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int seg = back ? sp.n - 1 - k - j : k + j;
            const bool in = k + j < sp.n;
            end[j] = in ? x[(int64_t)seg * cn] : 0.f;
            a[j] = in ? sum[(int64_t)seg * p.C] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (k + j >= sp.n) break;
            x[(int64_t)(back ? sp.n - 1 - k - j : k + j) * cn] = v;
            // (in two halves: where states grow, a segment's factor may pass the range although its product with a small
            // state does not; and nothing stays nothing, whatever the factor)
            const float half = exp2f(0.5f * A * a[j]);
            v = v == 0.f ? end[j] : fmaf(half * v, half, end[j]);
        }
    }
}

// The sums of the backward pass, each added in a fixed order. The first row_ctas CTAs: dB and dC from the tiles'
// parts; the others: dA, dD and ddt_bias from the segments'.
template <typename T>
__global__ void __launch_bounds__(256)
ssm_sums_kernel(const __grid_constant__ SsmProblem p, const Parts parts, const Tiles tl, int segs, unsigned row_ctas) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    float s = 0.f;
    if (blockIdx.x < row_ctas) {
        const int NP = (p.N + 3) / 4 * 4, wide = 2 * NP;
        const int64_t rows = p.B * p.T, id = (int64_t)blockIdx.x * 256 + threadIdx.x, k = id / wide;
        const int j = (int)(id - k * wide), n = j % NP;
        const int64_t row = k / p.G, g = k - row * p.G;
        if (row >= rows || n >= p.N) return;
        const float *at = parts.rows + (g * tl.per_group * rows + row) * wide + j;
#pragma unroll 8
        for (int i = 0; i < tl.per_group; ++i) s += at[i * rows * wide];
        put(static_cast<T *>(j < NP ? p.dBm : p.dCm) + (row * p.G + g) * p.N + n, s);
    } else {
        const int64_t w = p.N + 2, id = (int64_t)(blockIdx.x - row_ctas) * 256 + threadIdx.x, c = id / w, n = id - c * w;
        if (c >= p.C) return;
        const float *at = parts.chan + id;
#pragma unroll 8
        for (int64_t b = 0; b < p.B * segs; ++b) s += at[b * p.C * w];
        if (n < p.N) p.dA[c * p.N + n] = s;
        else if (n == p.N) { if (p.dD) p.dD[c] = s; }
        else if (p.dbias) p.dbias[c] = s;
    }
}

// One token of each row on the pages of a pool. kLanes lanes (4 kLanes >= N) own a channel, four states each, and keep
// its row of A while they go through rows of the batch, kRows at a time: all that these need is on its way
// together, and the page numbers of the next ones. A row's step size and output are made by one of the lanes. The
// states are read and written once. Measured: 240 rows of 4096 channels of 16 states (134 MB) 32 us a call, 26 in a graph
// where the pool (75 MB) stays in L2, and 30, 4.5 TB/s, on pages anywhere in 2 GB; with the loads of a row behind
// those of the row before, 61 a call. A CTA loads, computes and stores in turn, so its loads pause while it
// computes: latency bounds it before HBM does.
template <typename T, int kLanes>
__global__ void __launch_bounds__(256, 3)
ssm_step_kernel(const __grid_constant__ SsmProblem p, int vec, unsigned int *err) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    constexpr int kRows = 4, kOwn = kLanes < kRows ? kRows / kLanes : 1;     // rows of a lane: l, l + kLanes, ...
    using Raw = typename Pack<T, 4>::raw;
    const int l = threadIdx.x % kLanes, n0 = 4 * l;
    const int64_t c = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
    const bool live = c < p.C;
    const int64_t cc = live ? c : 0, g = cc / (p.C / p.G);
    const bool whole = p.N % 4 == 0, mine = live && n0 < p.N;
    float A[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) A[j] = live && n0 + j < p.N ? scale_a(p.A[cc * p.N + n0 + j]) : 0.f;
    const float D = p.D ? p.D[cc] : 0.f, bias = p.dt_bias ? p.dt_bias[cc] : 0.f;
    const int rows = (int)p.B, P = (int)p.P;        // (at most 2^30)
    auto page_of = [&](int r) { return r >= rows ? -1 : p.slots ? p.slots[r] : r; };
    auto quad = [&](const SsmRows &m, int r) {              // four values of a row of B or C
        const T *q = static_cast<const T *>(m.p) + r * m.b + g * p.N + n0;
        if (vec) return *reinterpret_cast<const Raw *>(q);
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = n0 + j < p.N ? get(q + j) : 0.f;
        return Pack<T, 4>::pack(f);                         // (they are T's values: nothing is rounded)
    };
    const int step = (int)gridDim.y * kRows;
    int next[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) next[i] = page_of((int)blockIdx.y * kRows + i);
    // (the whole warp walks together: rows past the last one do nothing)
    for (int r0 = (int)blockIdx.y * kRows; r0 < rows; r0 += step) {
        float4 h[kRows];
        Raw Br[kRows], Cr[kRows];
        float u[kOwn], d[kOwn], z[kOwn];
        int page[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (next[i] >= P && c == 0 && l == 0) atomicOr(err, kDevErrPages);
            page[i] = next[i] < P ? next[i] : -1;
            h[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            Br[i] = Cr[i] = Raw{};
            if (page[i] >= 0 && mine) {
                const float *S = p.S + ((int64_t)page[i] * p.C + cc) * p.N + n0;
                if (whole) {
                    h[i] = *reinterpret_cast<const float4 *>(S);
                } else {
                    h[i].x = S[0];
                    if (n0 + 1 < p.N) h[i].y = S[1];
                    if (n0 + 2 < p.N) h[i].z = S[2];
                    if (n0 + 3 < p.N) h[i].w = S[3];
                }
                Br[i] = quad(p.Bm, r0 + i);
                Cr[i] = quad(p.Cm, r0 + i);
            }
        }
#pragma unroll
        for (int k = 0; k < kOwn; ++k) {
            const int i = l + k * kLanes;
            u[k] = d[k] = z[k] = 0.f;
            if (i < kRows && live && r0 + i < rows) {
                u[k] = get(static_cast<const T *>(p.u.p) + (r0 + i) * p.u.b + c);
                d[k] = get(static_cast<const T *>(p.dt.p) + (r0 + i) * p.dt.b + c);
                if (p.z.p) z[k] = get(static_cast<const T *>(p.z.p) + (r0 + i) * p.z.b + c);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) next[i] = page_of(r0 + step + i);
#pragma unroll
        for (int k = 0; k < kOwn; ++k) d[k] = step_size<T>(d[k] + bias, p.softplus);
        float y[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const float di = __shfl_sync(0xffffffffu, d[i / kLanes], i % kLanes, kLanes);
            const float x = di * __shfl_sync(0xffffffffu, u[i / kLanes], i % kLanes, kLanes);
            float4 v;
            float Bv[4], Cv[4];
            Pack<T, 4>::unpack(Br[i], Bv);
            Pack<T, 4>::unpack(Cr[i], Cv);
            v.x = fmaf(ex2(fmaf(A[0], di, 2e-8f)), h[i].x, x * Bv[0]);
            v.y = fmaf(ex2(fmaf(A[1], di, 2e-8f)), h[i].y, x * Bv[1]);
            v.z = fmaf(ex2(fmaf(A[2], di, 2e-8f)), h[i].z, x * Bv[2]);
            v.w = fmaf(ex2(fmaf(A[3], di, 2e-8f)), h[i].w, x * Bv[3]);
            y[i] = fmaf(v.x, Cv[0], v.y * Cv[1]) + fmaf(v.z, Cv[2], v.w * Cv[3]);
            if (page[i] < 0 || !mine) y[i] = 0.f;       // (0 times an infinite d u is NaN)
            if (page[i] >= 0 && mine) {
                float *S = p.S + ((int64_t)page[i] * p.C + cc) * p.N + n0;
                if (whole) {
                    *reinterpret_cast<float4 *>(S) = v;
                } else {
                    S[0] = v.x;
                    if (n0 + 1 < p.N) S[1] = v.y;
                    if (n0 + 2 < p.N) S[2] = v.z;
                    if (n0 + 3 < p.N) S[3] = v.w;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (i % kLanes != l || !live || r0 + i >= rows) continue;
            float o = 0.f;
            if (page[i] >= 0) {
                o = y[i];
                if (p.D) o = fmaf(D, u[i / kLanes], o);
                if (p.z.p) o *= z[i / kLanes] * logistic<T>(z[i / kLanes]);
            }
            put(static_cast<T *>(p.o) + (int64_t)(r0 + i) * p.C + c, o);
        }
    }
}

// Shared memory of a ring (the kernels have up to 4 KB of their own).
constexpr size_t kRingBytes = 222 * 1024;

template <typename T, int kCh>
int ring_warps(const SsmProblem &p, int in, bool backward, int most) {
    const int64_t chunks = (p.T + kTok - 1) / kTok;
    int W = most;
    while (W > 1 && Ring<T, kCh>::bytes(W, in, p.N, p.row, backward) > kRingBytes) W -= W > 8 ? 4 : 1;
    return (int)std::min<int64_t>(W, chunks);
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

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
// The maps of a call (of its packed inputs); false where a map cannot be made.
bool make_maps(const SsmProblem &p, int ch, Maps *m) {
    const SsmRows *in[4] = {&p.u, &p.dt, &p.z, &p.go};
    void *const out[3] = {p.du ? p.du : p.o, p.ddt, p.dz};
    for (int i = 0; i < 4; ++i)
        if (in[i]->p && !rows_map(&m->in[i], in[i]->p, p.io, p.G * p.group, p.T, p.B, in[i]->t, in[i]->b, 32 * ch))
            return false;
    for (int i = 0; i < 3 && p.tma_out; ++i)
        if (out[i] && !rows_map(&m->out[i], out[i], p.io, p.C, p.T, p.B, p.C, p.T * p.C, 32 * ch)) return false;
    return rows_map(&m->b, p.Bm.p, p.io, p.G * p.row, p.T, p.B, p.Bm.t, p.Bm.b, p.row) &&
           rows_map(&m->c, p.Cm.p, p.io, p.G * p.row, p.T, p.B, p.Cm.t, p.Cm.b, p.row);
}

// TMA wants rows and tiles on 16 bytes. Inputs that are not (odd numbers of channels or states, slices that start
// anywhere) are first copied to rows that are: a copy costs a fraction of what reading them element by
// element did (16384 tokens of 3000 channels, B and C from an odd column on: 1190 us, 554 with the copy).
struct Packing {
    size_t bytes;               // of the copies
    bool copy[6];               // u, dt, z, go, B, C
};
// any: the most that pointers of any alignment need (of a forward call, or a backward one).
Packing packing_of(const SsmProblem &p, bool any, bool backward) {
    const int es = p.io == 0 ? 2 : 4, unit = 16 / es;
    const SsmRows *t[6] = {&p.u, &p.dt, &p.z, &p.go, &p.Bm, &p.Cm};
    const int64_t cg = p.C / p.G;
    Packing k{};
    for (int i = 0; i < 6; ++i) {
        const int64_t w = i < 4 ? cg : p.N;
        if (any ? i == 3 && !backward : !t[i]->p) continue;
        k.copy[i] = any || w % unit || reinterpret_cast<uintptr_t>(t[i]->p) % 16 || t[i]->b % unit || t[i]->t % unit ||
                    t[i]->b >= int64_t(1) << 38 || t[i]->t >= int64_t(1) << 38;     // (what a tensor map holds)
    }
    for (int i = 0; i < 6; ++i) {
        const int64_t w = i < 4 ? cg : p.N;
        if (k.copy[i]) k.bytes += round256((size_t)(p.B * p.T * p.G * ((w + unit - 1) / unit * unit)) * es);
    }
    return k;
}
struct PackJob {
    const void *from;
    int64_t b, t;               // element strides
    void *to;                   // [B, T, G, padded]
    int64_t width, padded;
};
struct PackJobs {
    PackJob job[6];
    int64_t T, rows;            // rows: B T G
    int G;
};
template <typename T>
__global__ void __launch_bounds__(256)
ssm_pack_kernel(const __grid_constant__ PackJobs jobs) {
    tc::pdl_launch_dependents();
    tc::pdl_wait_prerequisites();
    const PackJob &j = jobs.job[blockIdx.y];
    if (!j.to) return;
    T zero;
    put(&zero, 0.f);
    // a warp for a group of a token
    for (int64_t row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; row < jobs.rows; row += (int64_t)gridDim.x * 8) {
        const int64_t token = row / jobs.G, g = row - token * jobs.G, b = token / jobs.T, t = token - b * jobs.T;
        const T *from = static_cast<const T *>(j.from) + b * j.b + t * j.t + g * j.width;
        T *to = static_cast<T *>(j.to) + row * j.padded;
        for (int64_t i = threadIdx.x % 32; i < j.padded; i += 32) to[i] = i < j.width ? from[i] : zero;
    }
}
// Copies what has to be, and leaves the problem with inputs that TMA reads.
cudaError_t pack(SsmProblem *p, char *at, int num_sms, cudaStream_t s) {
    const Packing k = packing_of(*p, false, false);
    const int es = p->io == 0 ? 2 : 4, unit = 16 / es;
    const int64_t cg = p->C / p->G;
    SsmRows *t[6] = {&p->u, &p->dt, &p->z, &p->go, &p->Bm, &p->Cm};
    PackJobs jobs{};
    jobs.T = p->T;
    jobs.G = (int)p->G;
    jobs.rows = p->B * p->T * p->G;
    bool any = false;
    p->group = (cg + unit - 1) / unit * unit;
    p->row = (p->N + unit - 1) / unit * unit;
    p->tma_out = cg % unit == 0 && p->T * p->C < int64_t(1) << 38;
    for (int i = 0; i < 6; ++i) {
        if (!k.copy[i]) continue;
        any = true;
        const int64_t padded = i < 4 ? p->group : p->row;
        jobs.job[i] = PackJob{t[i]->p, t[i]->b, t[i]->t, at, i < 4 ? cg : p->N, padded};
        t[i]->p = at;
        t[i]->t = p->G * padded;
        t[i]->b = p->T * p->G * padded;
        at += round256((size_t)(jobs.rows * padded) * es);
    }
    if (!any) return cudaSuccess;
    const dim3 grid((unsigned)std::min<int64_t>((jobs.rows + 7) / 8, 8 * num_sms), 6);
    return launch(p->io == 0 ? ssm_pack_kernel<__nv_bfloat16> : ssm_pack_kernel<float>, grid, 256, 0, s, jobs);
}

// Channels of a lane in the backward pass: two share the loads of B and C and the sums across lanes (4 x 2047 tokens
// of 2048 channels, 16 states, bf16: 460 us against 585 with one), if a ring of eight warps still fits
// shared memory (2 x 358 tokens of 481 channels, 64 states: 672 us with two warps, 272 with one channel to a lane).
int bwd_channels(const SsmProblem &p) {
    const int unit = p.io == 0 ? 8 : 4, row = (p.N + unit - 1) / unit * unit;
    const size_t bytes = p.io == 0 ? Ring<__nv_bfloat16, 2>::bytes(8, 4, p.N, row, true)
                                   : Ring<float, 2>::bytes(8, 4, p.N, row, true);
    return bytes <= kRingBytes ? 2 : 1;
}

// Segments of a sequence for CTAs of 32 ch channels. Cutting it costs two thirds of a walk more (and the join), so it is
// done where the tiles leave more than half of the SMs idle; the segments then make one round of resident CTAs (two to
// an SM forward, one backward), or two rounds if those are better filled. Measured, 16384 tokens: forward, 512
// channels 88 us against 406 uncut, 2048 channels 330 against 408, 2560 channels 408 uncut against 481 in three;
// gradients, 1024 channels 575 us against 3266, 4864 channels of 8192 tokens 1216 against 1681.
Split split_of(const SsmProblem &p, int ch, bool backward, int splits, int num_sms) {
    const int64_t chunks = (p.T + kTok - 1) / kTok, ctas = p.B * tiles_of(p.C, p.G, ch).all;
    const int64_t round = backward ? num_sms : 2 * num_sms, most = chunks / (backward ? 16 : 8);
    int64_t n = 1;
    if (splits > 0) {
        n = std::min({(int64_t)splits, chunks, std::max<int64_t>(1, (int64_t(1) << 30) / ctas)});
    } else if (backward ? 2 * ctas <= num_sms : 9 * ctas <= 4 * num_sms) {
        const int64_t one = round / ctas, two = 2 * round / ctas;
        n = std::min(40 * two * ctas > 42 * 2 * one * ctas ? two : one, most);
    }
    if (p.B > 65535 || p.C * p.N > int64_t(1) << 30) n = 1;        // (the join's grid and indices)
    Split sp{};
    sp.chunks = (chunks + std::max<int64_t>(n, 1) - 1) / std::max<int64_t>(n, 1);
    sp.n = (int)((chunks + sp.chunks - 1) / sp.chunks);
    return sp;
}
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

template <typename T, int kCh, int kN, int kMode>
cudaError_t run_fwd(const SsmProblem &p, const Maps &maps, const Split &sp, int segs, int warps, float4 *marks,
                    unsigned int *err, cudaStream_t s) {
    constexpr int in = kMode == kOutputs ? 3 : 2;
    const int W = (int)std::min<int64_t>(ring_warps<T, kCh>(p, in, false, warps), sp.chunks);
    const size_t smem = Ring<T, kCh>::bytes(W, in, p.N, p.row, false);
    constexpr auto kernel = ssm_fwd_kernel<T, kCh, kN, kMode>;
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    return launch(kernel, dim3((unsigned)(p.B * segs * tiles_of(p.C, p.G, kCh).all)), 32 * W, smem, s, p, maps, sp,
                  segs, marks, err);
}
template <typename T, int kCh, int kMode>
cudaError_t fwd(const SsmProblem &p, const Maps &maps, const Split &sp, int segs, int num_sms, float4 *marks,
                unsigned int *err, cudaStream_t s) {
    // 16 warps to an SM: of one ring where there are no more rings than SMs
    const int warps = p.B * segs * tiles_of(p.C, p.G, kCh).all <= num_sms ? 16 : 8;
    if (p.N == 16) return run_fwd<T, kCh, 16, kMode>(p, maps, sp, segs, warps, marks, err, s);
    return run_fwd<T, kCh, 0, kMode>(p, maps, sp, segs, warps, marks, err, s);
}
cudaError_t join(const SsmProblem &p, const Split &sp, int directions, cudaStream_t s) {
    return launch(ssm_join_kernel, dim3((unsigned)((p.C * p.N + 255) / 256), directions, (unsigned)p.B), 256, 0, s, p,
                  sp);
}

template <typename T, int kCh, int kN, bool kEnd>
cudaError_t run_bwd(const SsmProblem &p, const Maps &maps, const Split &sp, const float4 *marks, const Parts &parts,
                    unsigned int *err, cudaStream_t s) {
    const int W = (int)std::min<int64_t>(ring_warps<T, kCh>(p, 4, true, kCh == 2 ? 8 : 12), sp.chunks);
    const size_t smem = Ring<T, kCh>::bytes(W, 4, p.N, p.row, true);
    constexpr auto kernel = ssm_bwd_kernel<T, kCh, kN, kEnd>;
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
    return launch(kernel, dim3((unsigned)(p.B * sp.n * tiles_of(p.C, p.G, kCh).all)), 32 * W, smem, s, p, maps, sp,
                  marks, parts, err);
}
template <typename T, int kCh, bool kEnd>
cudaError_t back(const SsmProblem &p, const Maps &maps, const Split &sp, const float4 *marks, const Parts &parts,
                 unsigned int *err, cudaStream_t s) {
    if (p.N == 16) return run_bwd<T, kCh, 16, kEnd>(p, maps, sp, marks, parts, err, s);
    return run_bwd<T, kCh, 0, kEnd>(p, maps, sp, marks, parts, err, s);
}

template <typename T>
cudaError_t whole_fwd(SsmProblem p, int splits, int num_sms, void *ws, unsigned int *err, cudaStream_t s) {
    Maps maps;
    Split sp = split_of(p, 1, false, splits, num_sms);
    p.stall = take_stall_hook() ? 1 : -1;
    char *at = static_cast<char *>(ws);
    const size_t copies = packing_of(p, false, false).bytes;
    cudaError_t e = pack(&p, at, num_sms, s);
    if (e == cudaSuccess && !make_maps(p, 1, &maps)) e = cudaErrorInvalidResourceHandle;
    if (e == cudaSuccess && sp.n > 1) {
        at += copies;
        sp.h = reinterpret_cast<float *>(at);
        sp.sum = reinterpret_cast<float *>(at + split_state_bytes(p, sp));
        // (nothing starts from the last one's end)
        e = fwd<T, 1, kEnds>(p, maps, sp, sp.n - 1, num_sms, nullptr, err, s);
        if (e == cudaSuccess) e = join(p, sp, 1, s);
    }
    if (e != cudaSuccess) return e;
    return fwd<T, 1, kOutputs>(p, maps, sp, sp.n, num_sms, nullptr, err, s);
}
template <typename T, int kCh>
cudaError_t whole_bwd(SsmProblem p, int splits, int num_sms, void *ws, unsigned int *err, cudaStream_t s) {
    Maps maps;
    Split sp = split_of(p, kCh, true, splits, num_sms);
    p.stall = take_stall_hook() ? 1 : -1;
    const BwdWorkspace lay = bwd_workspace(p, sp);
    char *at = static_cast<char *>(ws);
    const size_t copies = packing_of(p, false, false).bytes;
    cudaError_t e = pack(&p, at, num_sms, s);
    if (e == cudaSuccess && !make_maps(p, kCh, &maps)) e = cudaErrorInvalidResourceHandle;
    at += copies;
    float4 *marks = reinterpret_cast<float4 *>(at);
    const Parts parts{reinterpret_cast<float *>(at + lay.marks), reinterpret_cast<float *>(at + lay.marks + lay.rows)};
    if (e == cudaSuccess && sp.n > 1) {
        at += lay.marks + lay.rows + lay.chan;
        sp.h = reinterpret_cast<float *>(at);
        sp.g = reinterpret_cast<float *>(at + split_state_bytes(p, sp));
        sp.sum = reinterpret_cast<float *>(at + 2 * split_state_bytes(p, sp));
        e = fwd<T, kCh, kEnds>(p, maps, sp, sp.n, num_sms, nullptr, err, s);
        if (e == cudaSuccess) e = back<T, kCh, true>(p, maps, sp, nullptr, parts, err, s);
        if (e == cudaSuccess) e = join(p, sp, 2, s);
    }
    if (e == cudaSuccess) e = fwd<T, kCh, kMarks>(p, maps, sp, sp.n, num_sms, marks, err, s);
    if (e == cudaSuccess) e = back<T, kCh, false>(p, maps, sp, marks, parts, err, s);
    if (e != cudaSuccess) return e;
    const int64_t rows = p.B * p.T * p.G * 2 * ((p.N + 3) / 4 * 4), chan = p.C * (p.N + 2);
    const unsigned row_ctas = (unsigned)((rows + 255) / 256), ctas = row_ctas + (unsigned)((chan + 255) / 256);
    return launch(ssm_sums_kernel<T>, dim3(ctas), 256, 0, s, p, parts, tiles_of(p.C, p.G, kCh), sp.n, row_ctas);
}

}  // namespace

size_t ssm_fwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms, bool any) {
    const Split sp = split_of(p, 1, false, splits, num_sms);
    return packing_of(p, any, false).bytes + split_state_bytes(p, sp) + split_sum_bytes(p, sp);
}
size_t ssm_bwd_workspace_bytes(const SsmProblem &p, int splits, int num_sms, bool any) {
    return packing_of(p, any, true).bytes + bwd_workspace(p, split_of(p, bwd_channels(p), true, splits, num_sms)).all;
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

template <typename T, int kLanes>
static cudaError_t run_step(const SsmProblem &p, int num_sms, unsigned int *err, cudaStream_t s) {
    const int64_t tiles = (p.C * kLanes + 255) / 256, rows = (p.B + 3) / 4;
    // two rounds of resident CTAs, each with as many rows of its channels as that leaves
    const dim3 grid((unsigned)tiles, (unsigned)std::min<int64_t>(rows, std::max<int64_t>(1, 6 * num_sms / tiles)));
    const int vec = p.N % 4 == 0 && p.Bm.b % 4 == 0 && p.Cm.b % 4 == 0 &&
                    (reinterpret_cast<uintptr_t>(p.Bm.p) | reinterpret_cast<uintptr_t>(p.Cm.p)) % (4 * sizeof(T)) == 0;
    return launch(ssm_step_kernel<T, kLanes>, grid, 256, 0, s, p, vec, err);
}
template <typename T>
static cudaError_t step_of(const SsmProblem &p, int num_sms, unsigned int *err, cudaStream_t s) {
    if (p.N <= 4) return run_step<T, 1>(p, num_sms, err, s);
    if (p.N <= 8) return run_step<T, 2>(p, num_sms, err, s);
    if (p.N <= 16) return run_step<T, 4>(p, num_sms, err, s);
    if (p.N <= 32) return run_step<T, 8>(p, num_sms, err, s);
    if (p.N <= 64) return run_step<T, 16>(p, num_sms, err, s);
    return run_step<T, 32>(p, num_sms, err, s);
}

cudaError_t launch_ssm_step(const SsmProblem &p, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    return p.io == 0 ? step_of<__nv_bfloat16>(p, num_sms, dev_err, s) : step_of<float>(p, num_sms, dev_err, s);
}

}  // namespace gla
