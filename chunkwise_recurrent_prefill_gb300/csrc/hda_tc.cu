// Linear attention with one decay per head on the tensor cores (sm_103a): TMA-staged tiles,
// tcgen05 MMAs with TMEM accumulators, fp32 state in TMEM, warp-specialised roles.
//
// One map serves the forward and the three gradients (hda_internal.h). Per chunk of n = 64
// tokens (fewer at the end), with l = e^decay and the state S before the chunk:
//     P   = (X Y^T) . M,                  M_ij = l^|i-j| for j <= i (j >= i reversed), else 0
//     out = P Z + diag(f) X S,            f_i = l^(i+1)      (reversed: l^(n-1-i))
//     S  <- l^n S + Y^T diag(u) Z,        u_j = l^(n-1-j)    (reversed: l^(j+1))
// Every factor is a power with an exponent >= 0, so for decays <= 0 none overflows, whatever
// their strength; a constant decay makes M, f and u the same in every chunk. The kernels work
// on the transposes (out^T = Z^T P^T + S^T X^T diag(f), S^T += (diag(u) Z)^T Y): the state and
// the output then have M = 128 lanes, and S^T is an A operand straight from TMEM.
//
// Roundings to bf16: the operands themselves are bf16. P is rounded once after the mask, S once
// per chunk for its product with X (both end in an output that is bf16 itself). diag(u) Z is
// carried as a sum of two bf16 parts (2^-16 of a value is lost), because it goes into the fp32
// state that the caller gets back: with one part hT would be off by 2^-9.
//
// When there are fewer heads than SMs, each head's chunks are split into segments:
//   hda_tc_state_kernel : pieces of the segments but the last -> their end state from zero, E
//   hda_tc_scan_kernel  : S_start(s + 1) = l^tokens(s) S_start(s) + E(s)
//   hda_tc_out_kernel   : each segment from its start state; the last one gives the final state
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "gla_internal.h"
#include "hda_internal.h"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace gla {
namespace {

using namespace tc;

constexpr int kC = 64;              // tokens of a chunk
constexpr int kMaxSplits = 256;
constexpr int kMaxPieces = 8;

// l^n = e^(n g): the product is formed in two parts, so that the result is good to a few 2^-24
// of itself (the rounding of n g alone would cost 2^-24 |n g|). 1 for n = 0, whatever g is.
__device__ __forceinline__ float decay_pow(float g, float n) {
    if (n == 0.f) return 1.f;
    const float p = n * g;
    if (!(p > -100.f)) return expf(p);      // below (or NaN): the correction has no meaning
    return expf(p) * (1.f + fmaf(n, g, -p));
}

// One map as the kernels see it.
struct TcLin {
    const float *init;      // state before the first token (seg 0), or null
    const float *start;     // start states of segments 1 .. splits - 1 of its state problem
    float *fin;
    void *out;
    int init_t;             // init is [z][x]
    int start_t;            // start is [z][x] (it belongs to the transposed map)
    int out_f32;
    int Dx, Dz;
    int hx, hy, hz;         // state heads per head of x, y, z
    float a_in, a_out;
    int rev;
};

struct TcArgs {
    TcLin lin[3];
    const float *decay;
    int64_t T;
    int n, H, nchunks, splits;
    int hint;               // L2: what the out kernel reads is not read again
    unsigned *err;
};

struct TcMaps {
    CUtensorMap x[3], y[3], z[3];
};

// Chunks of segment `seg`, in the order of the walk.
__host__ __device__ __forceinline__ int seg_bound(int seg, int nchunks, int splits) {
    return (int)((int64_t)seg * nchunks / splits);
}

// Chunk at position p of the walk, and its tokens.
__device__ __forceinline__ int walk_chunk(int p, int nchunks, int rev) {
    return rev ? nchunks - 1 - p : p;
}
__device__ __forceinline__ int chunk_tokens(int c, int64_t T) {
    const int64_t left = T - (int64_t)c * kC;
    return left < kC ? (int)left : kC;
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ uint32_t par(int use) { return (uint32_t)use & 1u; }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&out)[32]) {
    uint32_t r0[16], r1[16];
    tmem_ld16(taddr, r0);
    tmem_ld16(taddr + 16, r1);
    tmem_wait_ld();
    reg_fence(r0);
    reg_fence(r1);
#pragma unroll
    for (int x = 0; x < 16; ++x) {
        out[x] = __uint_as_float(r0[x]);
        out[16 + x] = __uint_as_float(r1[x]);
    }
}

// The tile [64 tokens][D] of one head: one or two 128B-swizzled boxes of 64 columns, 8 KB each.
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int D,
                                          int h, int t, int b, uint64_t pol) {
    tma_load_4d_hint(dst, m, bar, 0, h, t, b, pol);
    if (D > 64) tma_load_4d_hint(dst + 8192, m, bar, 64, h, t, b, pol);
}

// 16 bytes of Z (8 values of one token) times the token's factor, as two bf16 parts.
__device__ __forceinline__ void split8(uint4 v, float u, uint4 &hi, uint4 &lo) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4], l[4];
    const float2 uu = make_float2(u, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = mul2(unpack_bf16(w[i]), uu);
        h[i] = pack_bf16(p.x, p.y);
        const float2 r = unpack_bf16(h[i]);
        l[i] = pack_bf16(p.x - r.x, p.y - r.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// ======================================================================= output kernel
namespace om {
constexpr int NQ = 3;                            // stages of x, y, z tiles
constexpr uint32_t X = 0, Y = 16384, Z = 32768, STAGE = 49152;
constexpr uint32_t ZP = NQ * STAGE;              // two buffers of diag(u) Z: high, low part
constexpr uint32_t ZPSTAGE = 32768;
constexpr uint32_t P = ZP + 2 * ZPSTAGE;         // [64 x 64] bf16, 128B swizzle
constexpr uint32_t PW = P + 8192;                // [65] f32 powers l^0 .. l^64
constexpr uint32_t FA = PW + 320;                // [128] f32 output factors a_out f_i
constexpr uint32_t BAR = FA + 512;
constexpr uint32_t NBAR = 24;
constexpr uint32_t TSLOT = BAR + NBAR * 8;
constexpr uint32_t ALLOC = TSLOT + 16 + 1024;
static_assert(ALLOC <= 232448, "output kernel shared memory");
constexpr uint32_t COL_S = 0;                    // S^T fp32, 128 columns (lane z, column x)
constexpr uint32_t COL_SB = 128;                 // its bf16 snapshots, 2 x 64
constexpr uint32_t COL_P = 256;                  // X Y^T (M = 64 layout)
constexpr uint32_t COL_OI = 320;                 // S^T X^T
constexpr uint32_t COL_OA = 384;                 // Z^T P^T
}  // namespace om

// Barriers. Where a producer may run two phases ahead of a waiter, the phases alternate between
// two barriers (ZDONE, ZFREE, SBFREE); elsewhere the next phase needs the waiter's own arrival.
enum {
    QFULL = 0, QEMPTY = 3, ZDONE = 6, ZFREE = 8, SBFREE = 10, PFULL = 12, PFREE = 13, PBF = 14,
    SREADY = 15, UDONE = 16, OFULL = 17, OFREE = 18, FIN = 19,
};
constexpr int kOutWarps = 14;   // 0 TMA, 1 MMA, 2-5 output, 6-9 state, 10-13 P and diag(u) Z
constexpr int kOutThreads = kOutWarps * 32;

__global__ void __launch_bounds__(kOutThreads, 1)
hda_tc_out_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a) {
    using namespace om;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = align1024(smraw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + TSLOT);
    float *pw = reinterpret_cast<float *>(sm + PW);
    float *fa = reinterpret_cast<float *>(sm + FA);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the maps of one segment are neighbours: they read the same tiles
    const int li = blockIdx.x % a.n;
    const int seg = (blockIdx.x / a.n) % a.splits;
    const int bh = blockIdx.x / a.n / a.splits;
    const int b = bh / a.H, h = bh % a.H;
    const TcLin &m = a.lin[li];
    const int rev = m.rev, Dx = m.Dx, Dz = m.Dz;
    const int cb = seg_bound(seg, a.nchunks, a.splits);
    const int n = seg_bound(seg + 1, a.nchunks, a.splits) - cb;
    auto chunk = [&](int c) { return walk_chunk(cb + c, a.nchunks, rev); };
    const float g = a.decay[h];

    if (threadIdx.x < 128) {
        const int i = threadIdx.x;
        if (i <= kC) pw[i] = decay_pow(g, (float)i);
        // forwards f_i = l^(i+1); reversed f_i = l^(n-1-i) = entry i + 64 - n of l^63 .. l^0
        fa[i] = i >= kC ? 0.f : m.a_out * decay_pow(g, (float)(rev ? kC - 1 - i : i + 1));
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&bars[QFULL + i], 1);
            mbar_init(&bars[QEMPTY + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[ZDONE + i], 4);
            mbar_init(&bars[ZFREE + i], 1);
            mbar_init(&bars[SBFREE + i], 1);
        }
        mbar_init(&bars[PFULL], 1);
        mbar_init(&bars[PFREE], 4);
        mbar_init(&bars[PBF], 4);
        mbar_init(&bars[SREADY], 4);
        mbar_init(&bars[UDONE], 1);
        mbar_init(&bars[OFULL], 1);
        mbar_init(&bars[OFREE], 4);
        mbar_init(&bars[FIN], 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.x[li]);
        tma_prefetch_desc(&maps.y[li]);
        tma_prefetch_desc(&maps.z[li]);
    }
    if (warp == 1) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0) {
            const uint64_t pol = a.hint ? l2_policy_evict_first() : l2_policy_evict_normal();
            const uint32_t bytes = (uint32_t)(2 * Dx + Dz) * 2 * kC;
            int c = 0;
            for (; c < n; ++c) {
                const int s = c % NQ;
                if (c >= NQ && !mbar_wait(&bars[QEMPTY + s], par(c / NQ - 1))) {
                    ok = false;
                    break;
                }
                uint8_t *base = sm + s * STAGE;
                uint64_t *fb = &bars[QFULL + s];
                const int t = chunk(c) * kC;
                mbar_arrive_expect_tx(fb, bytes);
                load_tile(base + X, &maps.x[li], fb, Dx, h / m.hx, t, b, pol);
                load_tile(base + Y, &maps.y[li], fb, Dx, h / m.hy, t, b, pol);
                load_tile(base + Z, &maps.z[li], fb, Dz, h / m.hz, t, b, pol);
            }
            // never leave with a copy still landing in this CTA's shared memory
            for (int i = 0; i < NQ; ++i) {
                const int uses = c > i ? (c - 1 - i) / NQ + 1 : 0;
                if (uses > 0 && !mbar_wait(&bars[QFULL + i], par(uses - 1))) ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // Three groups per chunk, each issued once its inputs are ready:
        //   U(c): snapshot of S taken, S decayed, diag(u) Z written  -> S^T += (diag(u) Z)^T Y
        //   P(c): tiles landed, P(c - 1) read                        -> X Y^T
        //   O(c): P tile written, O(c - 1) read                      -> S^T X^T, Z^T P^T
        // Lane 0's view of the barriers decides for the warp; one elected lane issues.
        const uint32_t idP = idesc_bf16(64, 64, 0, 0);
        const uint32_t idU = idesc_bf16(128, Dx, 1, 1);
        const uint32_t idOa = idesc_bf16(128, 64, 1, 0);
        const uint32_t idOi = idesc_bf16(128, 64, 0, 0);
        const int kx = Dx / 16;
        int np = 0, nu = 0, no = 0;
        uint32_t idle = 0;
        uint64_t t_idle = 0;
        while (no < n) {
            bool prog = false;
            if (__shfl_sync(0xffffffffu, nu < n && mbar_test(&bars[SREADY], par(nu)) &&
                                             mbar_test(&bars[ZDONE + (nu & 1)], par(nu >> 1)), 0)) {
                tc_fence_after();
                const uint32_t y = smem_u32(sm + (nu % NQ) * STAGE + Y);
                const uint32_t zp = smem_u32(sm + ZP + (nu & 1) * ZPSTAGE);
                if (elect_one()) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(tm + COL_S, smem_desc(zp + part * 16384 + kk * 2048, 8192, 1024),
                                   smem_desc(y + kk * 2048, 8192, 1024), idU, 1);
                    mma_commit(&bars[UDONE]);
                    mma_commit(&bars[ZFREE + (nu & 1)]);
                }
                __syncwarp();
                ++nu;
                prog = true;
            }
            if (__shfl_sync(0xffffffffu, np < n && mbar_test(&bars[QFULL + np % NQ], par(np / NQ)) &&
                                             (np == 0 || mbar_test(&bars[PFREE], par(np - 1))), 0)) {
                tc_fence_after();
                const uint32_t base = smem_u32(sm + (np % NQ) * STAGE);
                if (elect_one()) {
                    for (int x = 0; x < kx; ++x) {
                        const uint32_t off = (x >> 2) * 8192 + (x & 3) * 32;
                        mma_ss(tm + COL_P, smem_desc(base + X + off, 16, 1024),
                               smem_desc(base + Y + off, 16, 1024), idP, x > 0);
                    }
                    mma_commit(&bars[PFULL]);
                }
                __syncwarp();
                ++np;
                prog = true;
            }
            if (__shfl_sync(0xffffffffu, no < nu && mbar_test(&bars[PBF], par(no)) &&
                                             (no == 0 || mbar_test(&bars[OFREE], par(no - 1))), 0)) {
                tc_fence_after();
                const uint32_t base = smem_u32(sm + (no % NQ) * STAGE);
                const uint32_t pt = smem_u32(sm + P);
                if (elect_one()) {
                    for (int x = 0; x < kx; ++x)
                        mma_ts(tm + COL_OI, tm + COL_SB + (no & 1) * 64 + x * 8,
                               smem_desc(base + X + (x >> 2) * 8192 + (x & 3) * 32, 16, 1024), idOi,
                               x > 0);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(tm + COL_OA, smem_desc(base + Z + kk * 2048, 8192, 1024),
                               smem_desc(pt + kk * 32, 16, 1024), idOa, kk > 0);
                    mma_commit(&bars[OFULL]);
                    mma_commit(&bars[SBFREE + (no & 1)]);
                    // U(no) and P(no) were issued before: the stage has no reader left
                    mma_commit(&bars[QEMPTY + no % NQ]);
                }
                __syncwarp();
                ++no;
                prog = true;
            }
            if (prog) {
                idle = 0;
            } else {
                __nanosleep(32);    // leave the issue slots to the other warps
                if (++idle == 256) {
                    t_idle = global_ns();
                } else if ((idle & 1023) == 0 &&
                           __shfl_sync(0xffffffffu, global_ns() - t_idle > kWaitLimitNs, 0)) {
                    ok = false;
                    break;
                }
            }
        }
        // all issued MMAs complete before the CTA gives up its TMEM
        if (elect_one()) mma_commit(&bars[FIN]);
        __syncwarp();
        if (!mbar_wait(&bars[FIN], 0)) ok = false;
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------ output
        // Lane z of the accumulators, tokens in columns. A warp stores 32 neighbouring values
        // of one token at a time.
        const int j = warp & 3, z = j * 32 + lane;
        const uint64_t pol = l2_policy_evict_first();
        const int64_t rs = (int64_t)a.H * Dz;
        for (int c = 0; c < n; ++c) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[OFULL], par(c)))) { ok = false; break; }
            tc_fence_after();
            const int ch = chunk(c), nt = chunk_tokens(ch, a.T);
            const float *f = fa + (rev ? kC - nt : 0);
            float ov[64];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float oi[32], oa[32];
                tmem_ld32(tmem_addr(tm, j, COL_OI + 32 * half), oi);
                tmem_ld32(tmem_addr(tm, j, COL_OA + 32 * half), oa);
#pragma unroll
                for (int x = 0; x < 32; ++x) ov[32 * half + x] = fmaf(f[32 * half + x], oi[x], oa[x]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[OFREE]);
            if (z >= Dz) continue;
            const int64_t at = (((int64_t)b * a.T + (int64_t)ch * kC) * a.H + h) * Dz + z;
            if (m.out_f32) {
                float *op = static_cast<float *>(m.out) + at;
#pragma unroll
                for (int x = 0; x < kC; ++x)
                    if (x < nt) op[x * rs] = ov[x];
            } else {
                __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(m.out) + at;
                if (nt == kC) {
#pragma unroll
                    for (int x = 0; x < kC; ++x)
                        st_global_bf16_hint(op + x * rs, __float2bfloat16_rn(ov[x]), pol);
                } else {
#pragma unroll
                    for (int x = 0; x < kC; ++x)
                        if (x < nt) st_global_bf16_hint(op + x * rs, __float2bfloat16_rn(ov[x]), pol);
                }
            }
        }
        __syncwarp();
    } else if (warp < 10) {
        // ------------------------------------------------------------ state
        // Per chunk: the bf16 snapshot of S for X S, and S <- l^n S before the update is added.
        const int j = warp & 3, z = j * 32 + lane;
        const float *init = nullptr;
        int tr = 0;
        if (seg > 0) {
            // the start states come from the scan kernel, which may still be running
            pdl_wait_prerequisites();
            init = m.start + ((size_t)bh * (a.splits - 1) + (seg - 1)) * (Dx * Dz);
            tr = m.start_t;
        } else if (m.init) {
            init = m.init + (size_t)bh * Dx * Dz;
            tr = m.init_t;
        }
        const int sx = tr ? 1 : Dz, sz = tr ? Dx : 1;   // strides of the state as stored
#pragma unroll 1
        for (int x0 = 0; x0 < Dx; x0 += 16) {
            uint32_t r[16];
#pragma unroll
            for (int x = 0; x < 16; ++x)
                r[x] = (init && z < Dz) ? __float_as_uint(init[(x0 + x) * sx + z * sz]) : 0u;
            tmem_st16(tmem_addr(tm, j, COL_S + x0), r);
        }
        tmem_wait_st();
        for (int c = 0; c < n; ++c) {
            const bool w = (c == 0 || mbar_wait(&bars[UDONE], par(c - 1))) &&
                           (c < 2 || mbar_wait(&bars[SBFREE + (c & 1)], par((c >> 1) - 1)));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            tc_fence_after();
            const float carry = pw[chunk_tokens(chunk(c), a.T)];
            const float2 cc = make_float2(carry, carry);
#pragma unroll 1
            for (int q = 0; q < Dx / 32; ++q) {
                float sv[32];
                tmem_ld32(tmem_addr(tm, j, COL_S + 32 * q), sv);
                uint32_t pk[16], r0[16], r1[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) pk[x] = pack_bf16(sv[2 * x], sv[2 * x + 1]);
                tmem_st16(tmem_addr(tm, j, COL_SB + (c & 1) * 64 + 16 * q), pk);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float2 lo = mul2(make_float2(sv[2 * x], sv[2 * x + 1]), cc);
                    const float2 hi = mul2(make_float2(sv[16 + 2 * x], sv[17 + 2 * x]), cc);
                    r0[2 * x] = __float_as_uint(lo.x);
                    r0[2 * x + 1] = __float_as_uint(lo.y);
                    r1[2 * x] = __float_as_uint(hi.x);
                    r1[2 * x + 1] = __float_as_uint(hi.y);
                }
                tmem_st16(tmem_addr(tm, j, COL_S + 32 * q), r0);
                tmem_st16(tmem_addr(tm, j, COL_S + 32 * q + 16), r1);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SREADY]);
        }
        if (ok && m.fin && seg == a.splits - 1) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[UDONE], par(n - 1)))) {
                ok = false;
            } else {
                tc_fence_after();
                float *fp = m.fin + (size_t)bh * Dx * Dz + z;
#pragma unroll 1
                for (int q = 0; q < Dx / 32; ++q) {
                    float sv[32];
                    tmem_ld32(tmem_addr(tm, j, COL_S + 32 * q), sv);
                    if (z < Dz) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) fp[(32 * q + x) * Dz] = sv[x];
                    }
                }
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ diag(u) Z, then P
        const int j = warp & 3, ct = (warp - 10) * 32 + lane;
        // The warp's 16 rows of P over all 32 threads: rows ia and ia + 8, column pairs
        // 8 k + 2 (lane % 4). Their mask is the same in every chunk and stays in registers.
        const int ia = 16 * j + (lane >> 2), c0 = 2 * (lane & 3);
        float mask[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            const int i = ia + (e & 2 ? 8 : 0), col = 8 * (e >> 2) + c0 + (e & 1);
            const int d = rev ? col - i : i - col;
            mask[e] = d >= 0 ? m.a_in * m.a_out * pw[d] : 0.f;
        }
        // 16-byte vectors ct + 128 x of the Z tile: token (ct / 8 + 16 x) % 64
        const int row = ct >> 3;
        for (int c = 0; c < n; ++c) {
            const int s = c % NQ, nt = chunk_tokens(chunk(c), a.T);
            bool w = mbar_wait(&bars[QFULL + s], par(c / NQ)) &&
                     (c < 2 || mbar_wait(&bars[ZFREE + (c & 1)], par((c >> 1) - 1)));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            const uint4 *zs = reinterpret_cast<const uint4 *>(sm + s * STAGE + Z) + ct;
            uint4 *zh = reinterpret_cast<uint4 *>(sm + ZP + (c & 1) * ZPSTAGE) + ct;
            float u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int t = row + 16 * x, e = rev ? t + 1 : nt - 1 - t;
                u[x] = t < nt ? m.a_in * pw[e] : 0.f;
            }
#pragma unroll 1
            for (int box = 0; box < Dz / 64; ++box) {
                uint4 v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = zs[box * 512 + 128 * x];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint4 hi, lo;
                    split8(v[x], u[x], hi, lo);
                    zh[box * 512 + 128 * x] = hi;
                    zh[1024 + box * 512 + 128 * x] = lo;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[ZDONE + (c & 1)]);

            w = mbar_wait(&bars[PFULL], par(c)) && (c == 0 || mbar_wait(&bars[OFULL], par(c - 1)));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            tc_fence_after();
            uint32_t r0[16], r1[16];
            const uint32_t ta = tmem_addr(tm, j, COL_P);
            tmem_ld16x256b_x4(ta, r0);
            tmem_ld16x256b_x4(ta + 32, r1);
            tmem_wait_ld();
            reg_fence(r0);
            reg_fence(r1);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[PFREE]);
            uint8_t *pt = sm + P;
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) {
                const uint32_t *r = k8 < 4 ? r0 + 4 * k8 : r1 + 4 * (k8 - 4);
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float mk = mask[4 * k8 + e];
                    // a score outside the mask is dropped, not multiplied by zero: it may be
                    // infinite
                    f[e] = mk != 0.f ? mk * __uint_as_float(r[e]) : 0.f;
                }
                const int col = 8 * k8 + c0;
                *reinterpret_cast<uint32_t *>(pt + sw128_offset(ia, col)) = pack_bf16(f[0], f[1]);
                *reinterpret_cast<uint32_t *>(pt + sw128_offset(ia + 8, col)) = pack_bf16(f[2], f[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[PBF]);
        }
        __syncwarp();
    }

    if (!ok) atomicOr(a.err, kDevErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ======================================================================= state kernel
namespace st {
constexpr int NS = 4;
constexpr uint32_t Y = 0, Z = 16384, L = 32768, STAGE = 49152;   // L: low part of diag(u) Z
constexpr uint32_t PW = NS * STAGE;
constexpr uint32_t BAR = PW + 320;
constexpr uint32_t NBAR = 3 * NS + 1;
constexpr uint32_t TSLOT = BAR + NBAR * 8;
constexpr uint32_t ALLOC = TSLOT + 24 + 1024;
static_assert(ALLOC <= 232448, "state kernel shared memory");
}  // namespace st
enum { SFULL = 0, SEMPTY = st::NS, SZDONE = 2 * st::NS, SEND = 3 * st::NS };
constexpr int kStateThreads = 320;   // 0 TMA, 1 MMA, 2-9 diag(u) Z

struct StateProblem {
    float *E;               // [BH][(splits - 1) pieces][Dx][Dz]
    float *start;           // [BH][splits - 1][Dx][Dz]
    int li;                 // the map whose y and z it reads
};
struct StateArgs {
    StateProblem s[2];
    int n, pieces;
    int retain;             // chunks of a CTA (read last) that stay in L2 for the out kernel
};

// Chunks of piece `sub` of segment `seg`, in the order of the walk.
__device__ __forceinline__ void piece_range(const TcArgs &a, int seg, int sub, int pieces, int &cb,
                                            int &ce) {
    const int s0 = seg_bound(seg, a.nchunks, a.splits);
    const int len = seg_bound(seg + 1, a.nchunks, a.splits) - s0;
    cb = s0 + (int)((int64_t)sub * len / pieces);
    ce = s0 + (int)((int64_t)(sub + 1) * len / pieces);
}

__global__ void __launch_bounds__(kStateThreads, 1)
hda_tc_state_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a,
                    const __grid_constant__ StateArgs sa) {
    using namespace st;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = align1024(smraw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + TSLOT);
    float *pw = reinterpret_cast<float *>(sm + PW);
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int npc = (a.splits - 1) * sa.pieces;
    const int si = blockIdx.x % sa.n, pi = (blockIdx.x / sa.n) % npc, bh = blockIdx.x / sa.n / npc;
    const StateProblem &sp = sa.s[si];
    const TcLin &m = a.lin[sp.li];
    const int b = bh / a.H, h = bh % a.H, rev = m.rev, Dx = m.Dx, Dz = m.Dz;
    int cb, ce;
    piece_range(a, pi / sa.pieces, pi % sa.pieces, sa.pieces, cb, ce);
    const int n = ce - cb;
    // the chunks run last to first: what is read last is what the out kernel reads first
    auto chunk = [&](int c) { return walk_chunk(ce - 1 - c, a.nchunks, rev); };
    const float g = a.decay[h];
    if (threadIdx.x <= kC) pw[threadIdx.x] = decay_pow(g, (float)threadIdx.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[SFULL + i], 1);
            mbar_init(&bars[SEMPTY + i], 1);
            mbar_init(&bars[SZDONE + i], 8);
        }
        mbar_init(&bars[SEND], 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.y[sp.li]);
        tma_prefetch_desc(&maps.z[sp.li]);
    }
    if (warp == 1) tmem_alloc(tslot, 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_last(), drop = l2_policy_evict_first();
            int c = 0;
            for (; c < n; ++c) {
                const int s = c % NS;
                if (c >= NS && !mbar_wait(&bars[SEMPTY + s], par(c / NS - 1))) { ok = false; break; }
                uint8_t *base = sm + s * STAGE;
                const uint64_t pol = c >= n - sa.retain ? keep : drop;
                mbar_arrive_expect_tx(&bars[SFULL + s], (uint32_t)(Dx + Dz) * 2 * kC);
                load_tile(base + Y, &maps.y[sp.li], &bars[SFULL + s], Dx, h / m.hy, chunk(c) * kC, b, pol);
                load_tile(base + Z, &maps.z[sp.li], &bars[SFULL + s], Dz, h / m.hz, chunk(c) * kC, b, pol);
            }
            for (int i = 0; i < NS; ++i) {
                const int uses = c > i ? (c - 1 - i) / NS + 1 : 0;
                if (uses > 0 && !mbar_wait(&bars[SFULL + i], par(uses - 1))) ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idU = idesc_bf16(128, Dx, 1, 1);
        for (int c = 0; c < n; ++c) {
            const bool w = mbar_wait(&bars[SZDONE + c % NS], par(c / NS));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            tc_fence_after();
            const uint32_t base = smem_u32(sm + (c % NS) * STAGE);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(tm, smem_desc(base + (part ? L : Z) + kk * 2048, 8192, 1024),
                               smem_desc(base + Y + kk * 2048, 8192, 1024), idU,
                               (c > 0 || part > 0 || kk > 0) ? 1u : 0u);
                mma_commit(&bars[SEMPTY + c % NS]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&bars[SEND]);
        __syncwarp();
        if (!mbar_wait(&bars[SEND], 0)) ok = false;
        __syncwarp();
    } else {
        const int ct = (warp - 2) * 32 + lane;      // 0..255
        const int row = ct >> 3;                    // tokens row and row + 32
        for (int c = 0; c < n; ++c) {
            const int s = c % NS;
            if (!__all_sync(0xffffffffu, mbar_wait(&bars[SFULL + s], par(c / NS)))) { ok = false; break; }
            // c chunks of 64 tokens follow this one in the piece
            const float after = m.a_in * decay_pow(g, (float)(kC * c));
            const int nt = chunk_tokens(chunk(c), a.T);
            float u[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int t = row + 32 * x;
                u[x] = t < nt ? after * pw[rev ? t + 1 : nt - 1 - t] : 0.f;
            }
            uint4 *zs = reinterpret_cast<uint4 *>(sm + s * STAGE + Z) + ct;
#pragma unroll 1
            for (int box = 0; box < Dz / 64; ++box) {
                const uint4 v0 = zs[box * 512], v1 = zs[box * 512 + 256];
                uint4 hi, lo;
                split8(v0, u[0], hi, lo);
                zs[box * 512] = hi;
                zs[1024 + box * 512] = lo;
                split8(v1, u[1], hi, lo);
                zs[box * 512 + 256] = hi;
                zs[1024 + box * 512 + 256] = lo;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SZDONE + s]);
        }
        if (warp < 6) {     // E^T (lane z, column x) -> E[x][z]
            const int j = warp & 3, z = j * 32 + lane;
            if (!ok || !__all_sync(0xffffffffu, mbar_wait(&bars[SEND], 0))) {
                ok = false;
            } else {
                tc_fence_after();
                float *ep = sp.E + ((size_t)bh * npc + pi) * (Dx * Dz) + z;
#pragma unroll 1
                for (int q = 0; q < Dx / 32; ++q) {
                    float sv[32];
                    tmem_ld32(tmem_addr(tm, j, 32 * q), sv);
                    if (z < Dz) {
#pragma unroll
                        for (int x = 0; x < 32; ++x) ep[(32 * q + x) * Dz] = sv[x];
                    }
                }
            }
        }
        __syncwarp();
    }
    if (!ok) atomicOr(a.err, kDevErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 128);
    }
}

// ======================================================================= scan kernel
// Start states of segments 1 .. splits - 1. A thread carries kScanPer elements of one head; the
// loads of a batch of pieces are issued together, so the chain costs one round trip per batch.
constexpr int kScanThreads = 256, kScanPer = 4, kScanBatch = 4;

__global__ void __launch_bounds__(kScanThreads)
hda_tc_scan_kernel(const __grid_constant__ TcArgs a, const __grid_constant__ StateArgs sa) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const StateProblem &sp = sa.s[blockIdx.z];
    const TcLin &m = a.lin[sp.li];
    const int dd = m.Dx * m.Dz, e0 = blockIdx.y * (kScanThreads * kScanPer) + threadIdx.x;
    if (e0 >= dd) return;       // (dd is a multiple of a block's elements)
    const size_t bh = blockIdx.x;
    const float g = a.decay[bh % a.H];
    const int nseg = a.splits - 1, npc = nseg * sa.pieces;
    float s[kScanPer];
#pragma unroll
    for (int i = 0; i < kScanPer; ++i) {
        const int e = e0 + i * kScanThreads, x = e / m.Dz, z = e % m.Dz;
        s[i] = m.init ? m.init[bh * dd + (m.init_t ? z * m.Dx + x : e)] : 0.f;
    }
    const float *Eb = sp.E + bh * npc * dd + e0;
    float *ob = sp.start + bh * nseg * dd + e0;
    for (int r0 = 0; r0 < npc; r0 += kScanBatch) {
        float ev[kScanBatch][kScanPer];
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j)
            if (r0 + j < npc)
#pragma unroll
                for (int i = 0; i < kScanPer; ++i)
                    ev[j][i] = Eb[(size_t)(r0 + j) * dd + i * kScanThreads];
#pragma unroll
        for (int j = 0; j < kScanBatch; ++j) {
            if (r0 + j >= npc) break;
            const int r = r0 + j;
            int cb, ce;
            piece_range(a, r / sa.pieces, r % sa.pieces, sa.pieces, cb, ce);
            // only the first chunk of a reversed walk can be short
            int64_t tokens = (int64_t)(ce - cb) * kC;
            if (m.rev && cb == 0 && ce > 0) tokens -= kC - chunk_tokens(a.nchunks - 1, a.T);
            const float f = decay_pow(g, (float)tokens);
            const bool end = (r + 1) % sa.pieces == 0;
#pragma unroll
            for (int i = 0; i < kScanPer; ++i) {
                s[i] = fmaf(f, s[i], ev[j][i]);
                if (end) ob[(size_t)((r + 1) / sa.pieces - 1) * dd + i * kScanThreads] = s[i];
            }
        }
    }
}

// ======================================================================= host
constexpr int kMaxDevices = 64;
std::mutex g_attr_mu;
bool g_attr_done[kMaxDevices];

cudaError_t set_attrs() {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_attr_mu);
    if (g_attr_done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute((const void *)hda_tc_out_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, om::ALLOC);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute((const void *)hda_tc_state_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, st::ALLOC);
    if (e != cudaSuccess) return e;
    g_attr_done[dev] = true;
    return cudaSuccess;
}

bool make_map(CUtensorMap *m, const HdaTensor &t, int64_t B, int64_t T, int D) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)t.heads, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)t.h * 2, (cuuint64_t)t.t * 2, (cuuint64_t)t.b * 2};
    cuuint32_t box[4] = {64, 1, kC, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(t.p), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Maps whose states are computed apart: the forward's own; of the gradients, dq's (S^T) and
// dv's (dS), whose transpose serves dk.
int state_problems(const HdaProblem &p) { return p.n == 1 ? 1 : 2; }

// Segments per head and pieces per segment of the state pass. One out CTA runs per SM, so a
// call takes as many rounds of segments as there are CTAs per SM, rounded up, each with about
// two chunk times of start and end; the state pass costs about half a chunk time per chunk it
// reads, over all SMs, and a few more for itself and the scan.
int auto_splits(const HdaProblem &p, int sms) {
    const int64_t nchunks = (p.T + kC - 1) / kC, ctas = p.B * p.H * p.n;
    int best = 1;
    double least = 0;
    for (int64_t s = 1; s <= std::min<int64_t>(nchunks, kMaxSplits); ++s) {
        const double rounds = (double)((ctas * s + sms - 1) / sms);
        double cost = rounds * ((double)((nchunks + s - 1) / s) + 2.0);
        if (s > 1)
            cost += 4.0 + 0.5 * state_problems(p) * (double)(p.B * p.H) * nchunks * (s - 1) / s / sms;
        if (s == 1 || cost < least) {
            least = cost;
            best = (int)s;
        }
        if (ctas * s > 16 * (int64_t)sms) break;
    }
    return best;
}
int clamp_splits(const HdaProblem &p, int splits, int sms) {
    if (splits <= 0) return auto_splits(p, sms);
    const int64_t nchunks = (p.T + kC - 1) / kC;
    return (int)std::max<int64_t>(1, std::min<int64_t>({(int64_t)splits, nchunks, kMaxSplits}));
}
int state_pieces(const HdaProblem &p, int splits, int sms) {
    if (splits <= 1) return 1;
    const int64_t nchunks = (p.T + kC - 1) / kC;
    int64_t k = sms / (p.B * p.H * state_problems(p) * (splits - 1));
    k = std::min<int64_t>(k, nchunks / (4 * (int64_t)splits));
    return (int)std::max<int64_t>(1, std::min<int64_t>(k, kMaxPieces));
}

}  // namespace

bool hda_tc_supported(const HdaProblem &p) {
    if (p.io != 0 || p.T < 1 || p.T >= (int64_t(1) << 30) || p.B * p.H * 3 >= (int64_t(1) << 22))
        return false;
    for (int i = 0; i < p.n; ++i) {
        const HdaLin &m = p.lin[i];
        if ((m.Dx != 64 && m.Dx != 128) || (m.Dz != 64 && m.Dz != 128)) return false;
        for (const HdaTensor *t : {&m.x, &m.y, &m.z})     // limits of a tensor map
            for (int64_t s : {t->b, t->t, t->h})
                if (s * 2 >= (int64_t(1) << 40)) return false;
    }
    return true;
}

size_t hda_tc_workspace_bytes(const HdaProblem &p, int splits, int num_sms) {
    const int s = clamp_splits(p, splits, num_sms);
    if (s <= 1) return 0;
    const size_t per = (size_t)(p.B * p.H) * (s - 1) * p.lin[0].Dx * p.lin[0].Dz * sizeof(float);
    return state_problems(p) * per * (1 + state_pieces(p, s, num_sms));
}

cudaError_t launch_hda_tc(const HdaProblem &p, int splits, int num_sms, void *ws,
                          unsigned int *dev_err, cudaStream_t stream) {
    cudaError_t e = set_attrs();
    if (e != cudaSuccess) return e;
    const int s = clamp_splits(p, splits, num_sms), ns = state_problems(p);
    const int pieces = state_pieces(p, s, num_sms);
    const int64_t bh = p.B * p.H;
    TcMaps maps{};
    TcArgs a{};
    a.decay = p.decay;
    a.T = p.T;
    a.n = p.n;
    a.H = (int)p.H;
    a.nchunks = (int)((p.T + kC - 1) / kC);
    a.splits = s;
    a.hint = p.n == 1;
    a.err = dev_err;
    for (int i = 0; i < p.n; ++i) {
        const HdaLin &m = p.lin[i];
        if (!make_map(&maps.x[i], m.x, p.B, p.T, m.Dx) || !make_map(&maps.y[i], m.y, p.B, p.T, m.Dx) ||
            !make_map(&maps.z[i], m.z, p.B, p.T, m.Dz))
            return cudaErrorInvalidResourceHandle;   // a tensor map could not be encoded
        const auto rep = [&](const HdaTensor &t) { return (int)(p.H / t.heads); };
        a.lin[i] = TcLin{m.init, nullptr, m.fin, m.out, m.init_t, 0, m.out_f32, m.Dx, m.Dz,
                         rep(m.x), rep(m.y), rep(m.z), m.a_in, m.a_out, m.rev};
    }
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    if (s > 1) {
        const size_t per = (size_t)bh * (s - 1) * p.lin[0].Dx * p.lin[0].Dz;
        StateArgs sa{};
        sa.n = ns;
        sa.pieces = pieces;
        sa.retain = 0;
        float *w = static_cast<float *>(ws);
        for (int i = 0; i < ns; ++i) {
            sa.s[i].li = 2 * i;
            sa.s[i].E = w;
            sa.s[i].start = w + per * pieces;
            w += per * (pieces + 1);
            a.lin[2 * i].start = sa.s[i].start;
        }
        if (p.n == 3) {
            a.lin[1].start = a.lin[2].start;
            a.lin[1].start_t = 1;
        }
        hda_tc_state_kernel<<<(unsigned)(bh * (s - 1) * pieces * ns), kStateThreads, st::ALLOC, stream>>>(
            maps, a, sa);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        // the scan and the output may be scheduled while their predecessor still runs, and wait
        // for it before they read what it wrote
        cudaLaunchConfig_t cfg{};
        const int dd = p.lin[0].Dx * p.lin[0].Dz;
        cfg.gridDim = dim3((unsigned)bh, dd / (kScanThreads * kScanPer), ns);
        cfg.blockDim = dim3(kScanThreads);
        cfg.stream = stream;
        cfg.attrs = pdl;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, hda_tc_scan_kernel, a, sa)) != cudaSuccess) return e;
        count_launches(2);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(bh * s * p.n));
    cfg.blockDim = dim3(kOutThreads);
    cfg.dynamicSmemBytes = om::ALLOC;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = s > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, hda_tc_out_kernel, maps, a);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gla
