// Linear attention with one decay per head on the tensor cores (sm_103a): TMA-staged tiles,
// tcgen05 MMAs with TMEM accumulators, fp32 state in TMEM, warp-specialised roles.
//
// One map serves the forward and the three gradients (hda_internal.h). Per chunk of n = 64
// tokens (fewer at the end of the walk), with l = e^decay and the state S before the chunk:
//     P   = (X Y^T) . M,                  M_ij = l^|i-j| for j <= i (j >= i reversed), else 0
//     out = P Z + diag(f) X S,            f_i = l^(i+1)      (reversed: l^(63-i))
//     S  <- l^n S + Y^T diag(u) Z,        u_j = l^(n-1-j)    (reversed: l^(j+1), less the rows
//                                                             that a short chunk lacks)
// A constant decay makes M, f and u the same in every chunk. The kernels work on the transposes
// (out^T = Z^T P^T + S^T X^T diag(f), S^T += (diag(u) Z)^T Y): the state and the output then have
// M = 128 lanes, and S^T is an A operand straight from TMEM.
//
// Both terms of the output share one accumulator: out = diag(F) ((P / F) Z + X S) with
// F_i = max(f_i, 2^-60). The scores' factors M_ij / F_i stay below 2^60 (every other factor is a
// power with an exponent >= 0), so no decay overflows; where F_i is not f_i, X S counts 2^-60
// instead of less, which no output's 2^-9 can tell.
//
// Roundings to bf16: the operands themselves are bf16. P is rounded once after the mask, and S once
// per chunk for its product with X; both end in an output that is bf16 itself. diag(u) Z goes into
// the state as a sum of bf16 parts of 8 bits each: two where only outputs read the state (2^-16 of a
// term is lost; one part, 2^-9, raised the outputs' rms error from 0.0023 to 0.0028 of them, where
// their own rounding is 0.0017), three where the state is returned in fp32 (nothing of 24 bits is
// lost; with two parts hT was off by 3e-6, with three by 3e-7).
//
// When there are fewer heads than SMs, each head's chunks are split into segments:
//   hda_tc_state_kernel : pieces of the segments -> their end state from zero, E (of the last
//                         segment only where the final state is wanted)
//   hda_tc_scan_kernel  : S_start(s + 1) = l^tokens(s) S_start(s) + E(s), and the final state
//   hda_tc_out_kernel   : each segment from its start state (unsplit, it gives the final state too)
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
constexpr float kLeastF = 0x1p-60f; // least output factor
constexpr int kMaxSplits = 256;
constexpr int kMaxPieces = 8;
constexpr int64_t kL2Keep = 64ll << 20;

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
    int seg_len, seg_more;  // chunks of a segment; the first seg_more have one more
    int hint;               // L2: what the out kernel reads is not read again
    unsigned *err;
};

struct TcMaps {
    CUtensorMap x[3], y[3], z[3];   // loads: boxes of 64 columns, 64 tokens
    CUtensorMap o[3];               // stores: boxes of 32 columns (make_out_map)
};

// First chunk of segment `seg`, in the order of the walk.
__device__ __forceinline__ int seg_bound(int seg, const TcArgs &a) {
    return seg * a.seg_len + min(seg, a.seg_more);
}

// Chunk p of the walk: its first token and how many it has. A reversed walk counts its chunks from
// the end, so that here too only the last one is short; its first rows, before token 0, are read
// as zeros.
__device__ __forceinline__ int chunk_start(int p, const TcArgs &a, int rev) {
    return rev ? (int)a.T - kC * (p + 1) : kC * p;
}
__device__ __forceinline__ int chunk_tokens(int p, const TcArgs &a) {
    const int left = (int)a.T - kC * p;
    return left < kC ? left : kC;
}
// u_j of a chunk of nt tokens, from the powers pw.
__device__ __forceinline__ float state_factor(const float *pw, int row, int nt, int rev) {
    const int e = rev ? row - (kC - nt) + 1 : nt - 1 - row;
    return (rev ? e > 0 : e >= 0) ? pw[e] : 0.f;
}

__device__ __forceinline__ uint8_t *align1024(uint8_t *p) {
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ uint32_t par(int use) { return (uint32_t)use & 1u; }

// Bounded wait (false after kWaitLimitNs). One short loop that looks at the clock every 256th try:
// it is inlined at forty places, and with mbar_wait's two loops and timer the output kernel had 150 KB
// of code, more than an SM's instruction cache; reading the timer at every wait that does not
// succeed at once cost the roles hundreds of cycles, too.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity) {
    uint64_t t0 = 0;
#pragma unroll 1
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 255u) != 0) continue;
        const uint64_t t = global_ns();
        if (t0 == 0) t0 = t;
        else if (t - t0 > kWaitLimitNs) return false;
    }
    return true;
}

// The tile [64 tokens][D] of one head: one or two 128B-swizzled boxes of 64 columns, 8 KB each.
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *m, uint64_t *bar, int D,
                                          int h, int t, int b, uint64_t pol) {
    tma_load_4d_hint(dst, m, bar, 0, h, t, b, pol);
    if (D > 64) tma_load_4d_hint(dst + 8192, m, bar, 64, h, t, b, pol);
}

// 16 bytes of Z (8 values of one token) times the token's factor, as kParts bf16 parts (the first
// to dst, the others to rest, 16 KB apart) that hold 8 of the product's 24 bits each. (Cut off, not
// rounded: the upper half of a float is a bf16, so a part is a byte permutation and what remains a
// subtraction.)
template <int kParts>
__device__ __forceinline__ void put_scaled(uint4 v, float u, uint4 *dst, uint4 *rest) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float2 p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = mul2(unpack_bf16(w[i]), make_float2(u, u));
#pragma unroll
    for (int part = 0; part < kParts; ++part) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __float_as_uint(p[i].x), y = __float_as_uint(p[i].y);
            o[i] = __byte_perm(x, y, 0x7632);
            if (part + 1 < kParts)
                p[i] = add2(p[i], make_float2(__uint_as_float((x & 0xffff0000u) ^ 0x80000000u),
                                              __uint_as_float((y & 0xffff0000u) ^ 0x80000000u)));
        }
        (part == 0 ? dst : rest + (part - 1) * 1024)[0] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ======================================================================= output kernel
namespace om {
constexpr int NQ = 3;                            // stages of x, y, z tiles
constexpr uint32_t X = 0, Y = 16384, Z = 32768, STAGE = 49152;
constexpr uint32_t ZP = NQ * STAGE;              // diag(u) Z, two or three parts
constexpr uint32_t P = ZP + 3 * 16384;           // two [64 x 64] bf16 tiles, 128B swizzle
constexpr uint32_t OUT = P + 2 * 8192;           // a [64 x 32] bf16 (or [32 x 32] f32) tile per warp
constexpr uint32_t PW = OUT + 4 * 4096;          // [65] f32 powers l^0 .. l^64
constexpr uint32_t FA = PW + 320;                // [64] f32 output factors a_out F_i
constexpr uint32_t FU = FA + 256;                // [64] f32 state factors a_in u_j of a full chunk
constexpr uint32_t FUL = FU + 256;               // the same of the last chunk of the walk
constexpr uint32_t MASK = FUL + 256;             // [128] f32 M_ij by i - j + 64
constexpr uint32_t BAR = MASK + 512;
constexpr uint32_t NBAR = 28;
constexpr uint32_t TSLOT = BAR + NBAR * 8;
constexpr uint32_t ALLOC = TSLOT + 16 + 1024;
static_assert(ALLOC <= 232448, "output kernel shared memory");
constexpr uint32_t COL_S = 0;                    // S^T fp32: lane z, column x
constexpr uint32_t COL_P = 256;                  // X Y^T (M = 64 layout)
constexpr uint32_t COL_O = 320;                  // S^T X^T + Z^T P^T: two of 64 columns
// the state's bf16 snapshots: two of 64 columns; with a returned state (kExact) one, further on,
// and a chunk's (diag(u) Z)^T Y apart from S
constexpr uint32_t COL_SB = 128, COL_SB_EXACT = 448, COL_D = 128;
}  // namespace om

// Barriers. Where a producer may run two phases ahead of a waiter, the phases alternate between
// the barriers of the buffers (PBF, OFULL, OFREE, IDONE); elsewhere the next phase needs the waiter's
// own arrival.
enum {
    QFULL = 0, QEMPTY = 3, PBF = 6, OFULL = 8, OFREE = 10, IDONE = 12, ZDONE = 14, ZFREE = 15, PFULL = 16,
    PFREE = 17, SREADY = 18, SBFREE = 19, UDONE = 20, FIN = 21,
};
static_assert(FIN < (int)om::NBAR, "output kernel barrier map");
// Warps: 0 TMA, 1 and 19 MMA, 2-5 output, 6-9 state, 10-13 P and the second box of diag(u) Z, 14-17 its
// first box (18: none). Every role has a loop of its own, since what it does in a chunk is mostly
// waiting: for barriers, fences, TMEM, and for shared memory, which the tiles' copies and the MMAs
// keep busy for 60 % of a chunk's time (240 KB of it).
// The loops are kept short, since different ones share the instruction cache of each quarter of the
// SM. 14 warps (roles joined), 22 and 28 warps (state and scaling spread out) were slower.
constexpr int kOutWarps = 20;
constexpr int kOutThreads = kOutWarps * 32;

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// 32 lanes x 32 columns of fp32 accumulators -> 32 floats.
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&out)[32]) {
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

// kExact: the state is returned from here (a sequence that is not split), so its updates take
// three parts of diag(u) Z, and each chunk's is accumulated by itself.
// CTA = one segment of one head and map (the maps of one segment are neighbours: they read the
// same tiles). The maps are lin[first] .. lin[first + count - 1].
// Measured at D = 128: 1.75 us a chunk, of which the tensor pipe is busy for 40 % and the shared
// memory's data pipe for 50 % (plus the copies' and MMAs' own reads): 16 heads of 16384 tokens 50 us
// (5.4 TB/s), their three gradients 131 us, 16 x 16 heads of 2501 tokens with returned states 153 us.
// (Two kernels, not two branches of one: an SM's instruction cache does not hold both.)
template <bool kExact>
__global__ void __launch_bounds__(kOutThreads, 1)
hda_tc_out_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a, const int first,
                  const int count) {
    using namespace om;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = align1024(smraw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + TSLOT);
    float *pw = reinterpret_cast<float *>(sm + PW);
    float *fa = reinterpret_cast<float *>(sm + FA);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    const int li = first + blockIdx.x % count;
    const int seg = (blockIdx.x / count) % a.splits;
    const int bh = blockIdx.x / count / a.splits;
    const int b = bh / a.H, h = bh % a.H;
    const TcLin &m = a.lin[li];
    const int rev = m.rev, Dx = m.Dx, Dz = m.Dz;
    const int cb = seg_bound(seg, a);
    const int n = seg_bound(seg + 1, a) - cb;
    const float g = a.decay[h];
    constexpr int kParts = kExact ? 3 : 2;
    constexpr uint32_t kColU = kExact ? COL_D : COL_S;

    if (threadIdx.x < 128) {
        const int i = threadIdx.x;
        if (i <= kC) pw[i] = decay_pow(g, (float)i);
        if (i < kC)
            fa[i] = m.a_out * fmaxf(decay_pow(g, (float)(rev ? kC - 1 - i : i + 1)), kLeastF);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < NQ; ++i) {
            mbar_init(&bars[QFULL + i], 1);
            mbar_init(&bars[QEMPTY + i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[PBF + i], 4);
            mbar_init(&bars[OFULL + i], 1);
            mbar_init(&bars[OFREE + i], 4);
            mbar_init(&bars[IDONE + i], 1);
        }
        mbar_init(&bars[ZDONE], 8);
        mbar_init(&bars[ZFREE], 1);
        mbar_init(&bars[PFULL], 1);
        mbar_init(&bars[PFREE], 4);
        mbar_init(&bars[SREADY], 4);
        mbar_init(&bars[SBFREE], 1);
        mbar_init(&bars[UDONE], 1);
        mbar_init(&bars[FIN], 2);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.x[li]);
        tma_prefetch_desc(&maps.y[li]);
        tma_prefetch_desc(&maps.z[li]);
        tma_prefetch_desc(&maps.o[li]);
    }
    if (warp == 1) tmem_alloc(tslot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x < 2 * kC) {     // the factors of a full chunk, then those of the last one
        const int i = threadIdx.x & (kC - 1);
        const int nt = threadIdx.x < kC ? kC : chunk_tokens(a.nchunks - 1, a);
        reinterpret_cast<float *>(sm + FU)[threadIdx.x] = m.a_in * state_factor(pw, i, nt, rev);
        const int d = rev ? kC - (int)threadIdx.x : (int)threadIdx.x - kC;
        reinterpret_cast<float *>(sm + MASK)[threadIdx.x] = d >= 0 ? pw[d] : 0.f;
    }
    __syncthreads();
    const uint32_t tm = *tslot;
    bool ok = true;
    const int j = warp & 3;     // the warp's quarter of the TMEM lanes

    // diag(u) Z of chunk c, boxes b0 .. b1 - 1 of 64 value columns, by four warps (ct: the thread).
    // 16-byte vectors ct + 128 x of a box: token (ct / 8 + 16 x) % 64. The product keeps the tile's
    // layout, so the swizzle does not matter here.
    auto scale_Z = [&](int c, int ct, int b0, int b1) -> bool {
        const int s = c % NQ;
        const bool w = wait_bar(&bars[QFULL + s], par(c / NQ)) &&
                       (c == 0 || wait_bar(&bars[ZFREE], par(c - 1)));
        if (!__all_sync(0xffffffffu, w)) return false;
        const float *u = reinterpret_cast<const float *>(sm + (cb + c == a.nchunks - 1 ? FUL : FU)) + (ct >> 3);
        const uint4 *zs = reinterpret_cast<const uint4 *>(sm + s * STAGE + Z) + ct;
        uint4 *zp = reinterpret_cast<uint4 *>(sm + ZP) + ct;
#pragma unroll 1
        for (int box = b0; box < b1; ++box) {
#pragma unroll 1
            for (int x0 = 0; x0 < 4; x0 += 2) {     // (two vectors at a time, for want of registers)
                uint4 v[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) v[x] = zs[box * 512 + 128 * (x0 + x)];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int at = box * 512 + 128 * (x0 + x);
                    put_scaled<kParts>(v[x], u[16 * (x0 + x)], zp + at, zp + 1024 + at);
                }
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[ZDONE]);
        return true;
    };

    if (warp == 0) {
        if (lane == 0) {
            // -------------------------------------------------------- TMA producer
            const uint64_t pol = a.hint ? l2_policy_evict_first() : l2_policy_evict_normal();
            const uint32_t bytes = (uint32_t)(2 * Dx + Dz) * 2 * kC;
            int c = 0;
            for (; c < n; ++c) {
                const int s = c % NQ;
                if (c >= NQ && !wait_bar(&bars[QEMPTY + s], par(c / NQ - 1))) {
                    ok = false;
                    break;
                }
                uint8_t *base = sm + s * STAGE;
                uint64_t *fb = &bars[QFULL + s];
                const int t = chunk_start(cb + c, a, rev);
                mbar_arrive_expect_tx(fb, bytes);
                load_tile(base + X, &maps.x[li], fb, Dx, h / m.hx, t, b, pol);
                load_tile(base + Y, &maps.y[li], fb, Dx, h / m.hy, t, b, pol);
                load_tile(base + Z, &maps.z[li], fb, Dz, h / m.hz, t, b, pol);
            }
            // never leave with a copy still landing in this CTA's shared memory
            for (int i = 0; i < NQ; ++i) {
                const int uses = c > i ? (c - 1 - i) / NQ + 1 : 0;
                if (uses > 0 && !wait_bar(&bars[QFULL + i], par(uses - 1))) ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1 || warp == 19) {
        // ------------------------------------------------------------ MMA issuers
        // Two warps, each with two groups per chunk in a fixed order that the other roles keep up
        // with (one warp that issued all four spent 2600 cycles a chunk on it, 1000 of them on
        // waits and commits one after another):
        //   1 : U(c)     S decayed, diag(u) Z written -> S += (diag(u) Z)^T Y
        //                (kExact: D(c - 1) read -> D = (diag(u) Z)^T Y, which the state warps add)
        //       I(c)     snapshot of S taken, out(c - 2) read -> O = S^T X^T
        //   19: P(c + 1) tiles landed, P(c) read -> X Y^T
        //       A(c)     I(c) complete, P tile written -> O += Z^T P^T
        // A stage is free once both have committed their last reads of it. A warp waits converged,
        // then one elected lane issues. The operand descriptors are made once: a tile further on
        // is an addition to the address field (in 16-byte units; the field does not overflow).
        const uint32_t s0 = smem_u32(sm);
        const uint64_t dX = smem_desc(s0 + X, 16, 1024), dY = smem_desc(s0 + Y, 16, 1024);
        // K-major operands: 16 columns of a 64-column box are 32 bytes, the boxes 8 KB apart
        auto koff = [](int x) { return (uint64_t)((x >> 2) * (8192 >> 4) + (x & 3) * (32 >> 4)); };
        const bool wide = Dx > 64;
        bool w;
        if (warp == 1) {
            const uint32_t idU = idesc_bf16(128, Dx, 1, 1), idOi = idesc_bf16(128, 64, 0, 0);
            const uint64_t dYt = smem_desc(s0 + Y, 8192, 1024), dZP = smem_desc(s0 + ZP, 8192, 1024);
            for (int c = 0, s = 0; c < n; ++c) {
                const uint64_t so = (uint64_t)(s * (STAGE >> 4));
                w = wait_bar(&bars[SREADY], par(c)) && wait_bar(&bars[ZDONE], par(c));
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t y0 = dYt + so;
                    // the small parts first: the accumulator drops the bits below its own last one
                    // at every step, so the fewer steps it is large in, the better
#pragma unroll
                    for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(tm + kColU, dZP + part * (16384 >> 4) + kk * (2048 >> 4),
                                   y0 + kk * (2048 >> 4), idU, !kExact || part < kParts - 1 || kk > 0);
                    mma_commit(&bars[UDONE]);
                    mma_commit(&bars[ZFREE]);
                }
                __syncwarp();
                w = c < 2 || wait_bar(&bars[OFREE + (c & 1)], par((c >> 1) - 1));
                if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t x0 = dX + so;
                    const uint32_t sb = tm + (kExact ? COL_SB_EXACT : COL_SB + (c & 1) * 64);
                    const uint32_t o = tm + COL_O + (c & 1) * 64;
#pragma unroll
                    for (int x = 0; x < 4; ++x) mma_ts(o, sb + x * 8, x0 + koff(x), idOi, x > 0);
                    if (wide) {
#pragma unroll
                        for (int x = 4; x < 8; ++x) mma_ts(o, sb + x * 8, x0 + koff(x), idOi, 1);
                    }
                    if (kExact) mma_commit(&bars[SBFREE]);
                    mma_commit(&bars[IDONE + (c & 1)]);
                    mma_commit(&bars[QEMPTY + s]);
                }
                __syncwarp();
                s = s + 1 == NQ ? 0 : s + 1;
            }
        } else {
            const uint32_t idP = idesc_bf16(64, 64, 0, 0), idOa = idesc_bf16(128, 64, 1, 0);
            const uint64_t dZt = smem_desc(s0 + Z, 8192, 1024), dP = smem_desc(s0 + P, 16, 1024);
            for (int c = -1, s = 0; c < n; ++c) {       // s: the stage of chunk c (0 for c = -1)
                const int s1 = c < 0 ? 0 : s + 1 == NQ ? 0 : s + 1;
                if (c + 1 < n) {
                    w = wait_bar(&bars[QFULL + s1], par((c + 1) / NQ)) && (c < 0 || wait_bar(&bars[PFREE], par(c)));
                    if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t x0 = dX + (uint64_t)(s1 * (STAGE >> 4)), y0 = dY + (uint64_t)(s1 * (STAGE >> 4));
#pragma unroll
                        for (int x = 0; x < 4; ++x) mma_ss(tm + COL_P, x0 + koff(x), y0 + koff(x), idP, x > 0);
                        if (wide) {
#pragma unroll
                            for (int x = 4; x < 8; ++x) mma_ss(tm + COL_P, x0 + koff(x), y0 + koff(x), idP, 1);
                        }
                        mma_commit(&bars[PFULL]);
                    }
                    __syncwarp();
                }
                if (c >= 0) {
                    w = wait_bar(&bars[PBF + (c & 1)], par(c >> 1)) && wait_bar(&bars[IDONE + (c & 1)], par(c >> 1));
                    if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t z0 = dZt + (uint64_t)(s * (STAGE >> 4)), p0 = dP + (uint64_t)((c & 1) * (8192 >> 4));
                        const uint32_t o = tm + COL_O + (c & 1) * 64;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ss(o, z0 + kk * (2048 >> 4), p0 + kk * (32 >> 4), idOa, 1);
                        mma_commit(&bars[OFULL + (c & 1)]);
                        mma_commit(&bars[QEMPTY + s]);
                    }
                    __syncwarp();
                }
                s = s1;
            }
        }
        // all issued MMAs complete before the CTA gives up its TMEM
        if (elect_one()) mma_commit(&bars[FIN]);
        __syncwarp();
        if (!wait_bar(&bars[FIN], 0)) ok = false;
        __syncwarp();
    } else if (warp < 6) {
        // ------------------------------------------------------------ output
        // out^T = O diag(F): lane z, tokens in columns. A warp stages its 32 value columns as
        // [token][32] rows (64 bytes, 16-byte chunks XORed with (row / 2) % 4), which one bulk
        // store then takes to global memory. (Loads in the mma fragment layout, whose transposing
        // stores need fewer instructions, took 2.5 times as long.)
        const int z = j * 32 + lane;
        const uint64_t pol = l2_policy_evict_first();
        uint8_t *tile = sm + OUT + j * 4096;
        const bool mine = 32 * j < Dz;      // this warp's columns exist
        uint32_t at[4];                     // of this lane in rows 2 r, 2 r + 1 modulo 8
#pragma unroll
        for (int r = 0; r < 4; ++r) at[r] = smem_u32(tile) + (((lane >> 3) ^ r) << 4) + (lane & 7) * 2;
        for (int c = 0; c < n; ++c) {
            if (!__all_sync(0xffffffffu, wait_bar(&bars[OFULL + (c & 1)], par(c >> 1)))) { ok = false; break; }
            tc_fence_after();
            const int t0 = chunk_start(cb + c, a, rev), nt = chunk_tokens(cb + c, a);
            const uint32_t ta = tmem_addr(tm, j, COL_O + (c & 1) * 64);
            const bool bulk = nt == kC;     // else row by row, straight from here
            if (mine && bulk) {
#pragma unroll 1
                for (int q = 0; q < kC; q += 16) {
                    // the staging tile has been read (it takes 64 tokens of bf16, 32 of float)
                    if (q == 0 || (m.out_f32 && q == 32)) {
                        if (lane == 0) bulk_wait_read_all();
                        __syncwarp();
                    }
                    uint32_t r[16];
                    tmem_ld16(ta + q, r);
                    float4 f[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) f[x] = *reinterpret_cast<const float4 *>(fa + q + 4 * x);
                    tmem_wait_ld();
                    reg_fence(r);
                    float2 v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        v[x] = mul2(make_float2(__uint_as_float(r[2 * x]), __uint_as_float(r[2 * x + 1])),
                                    x & 1 ? make_float2(f[x >> 1].z, f[x >> 1].w)
                                          : make_float2(f[x >> 1].x, f[x >> 1].y));
                    if (m.out_f32) {
                        float *to = reinterpret_cast<float *>(tile) + (q & 31) * 32 + lane;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            to[2 * x * 32] = v[x].x;
                            to[(2 * x + 1) * 32] = v[x].y;
                        }
                        if (q & 16) {
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) {
                                tma_store_4d_hint(&maps.o[li], tile, 32 * j, h, t0 + q - 16, b, pol);
                                bulk_commit();
                            }
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            asm volatile("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %0;\n\t"
                                         "st.shared.b16 [%1], lo;\n\tst.shared.b16 [%1 + 64], hi;\n\t}" ::"r"(
                                             pack_bf16(v[x].x, v[x].y)),
                                         "r"(at[x & 3] + (q + 2 * x) * 64)
                                         : "memory");
                    }
                }
            } else if (mine) {
                const int64_t rs = (int64_t)a.H * Dz;
                const int64_t base = ((int64_t)b * a.T + t0) * rs + (int64_t)h * Dz + z;
                const int lo = rev ? kC - nt : 0, hi = rev ? kC : nt;    // the rows there are
#pragma unroll 1
                for (int q = 0; q < kC; q += 8) {
                    uint32_t r[8];
                    tmem_ld8(ta + q, r);
                    tmem_wait_ld();
                    reg_fence(r);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const int row = q + x;
                        if (row < lo || row >= hi) continue;
                        const float v = fa[row] * __uint_as_float(r[x]);
                        if (m.out_f32) static_cast<float *>(m.out)[base + row * rs] = v;
                        else static_cast<__nv_bfloat16 *>(m.out)[base + row * rs] = __float2bfloat16_rn(v);
                    }
                }
            }
            tc_fence_before();
            const bool store = mine && bulk && !m.out_f32;
            if (store) fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars[OFREE + (c & 1)]);
                if (store) {
                    tma_store_4d_hint(&maps.o[li], tile, 32 * j, h, t0, b, pol);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else if (warp >= 10 && warp < 14) {
        // ------------------------------------------------------------ P
        // X Y^T of chunk c -> its masked bf16 tile. The tile's buffer was last read by A(c - 2),
        // which PFULL(c), whose MMAs were issued later, has seen complete. A warp has 16 rows: ia
        // and ia + 8 of a thread, column pairs 8 k + 2 (lane % 4). The factors are the same in every
        // chunk and stay in registers.
        const int ia = 16 * j + (lane >> 2), c0 = 2 * (lane & 3);
        float mask[32], rf[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
            rf[e] = m.a_in / fmaxf(pw[rev ? kC - 1 - ia - 8 * e : ia + 8 * e + 1], kLeastF);
        const float *mk = reinterpret_cast<const float *>(sm + MASK) + kC + ia - c0;
#pragma unroll
        for (int e = 0; e < 32; ++e)        // M_ij / F_i (a_out is in F, a_in here)
            mask[e] = mk[(e & 2 ? 8 : 0) - 8 * (e >> 2) - (e & 1)] * rf[(e >> 1) & 1];
        for (int c = 0; c < n; ++c) {
            // (the second box of diag(u) Z is these warps')
            if (!scale_Z(c, (warp - 10) * 32 + lane, 1, Dz / 64)) { ok = false; break; }
            if (!__all_sync(0xffffffffu, wait_bar(&bars[PFULL], par(c)))) { ok = false; break; }
            tc_fence_after();
            uint8_t *pt = sm + P + (c & 1) * 8192;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t r[16];
                tmem_ld16x256b_x4(tmem_addr(tm, j, COL_P + 32 * half), r);
                tmem_wait_ld();
                reg_fence(r);
                if (half == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[PFREE]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at = 16 * half + 4 * k + 2 * e;
                        f[e] = mul2(make_float2(mask[at], mask[at + 1]),
                                    make_float2(__uint_as_float(r[4 * k + 2 * e]),
                                                __uint_as_float(r[4 * k + 2 * e + 1])));
                    }
                    const int col = c0 + 32 * half + 8 * k;
                    *reinterpret_cast<uint32_t *>(pt + sw128_offset(ia, col)) = pack_bf16(f[0].x, f[0].y);
                    *reinterpret_cast<uint32_t *>(pt + sw128_offset(ia + 8, col)) = pack_bf16(f[1].x, f[1].y);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[PBF + (c & 1)]);
        }
        __syncwarp();
    } else if (warp >= 14 && warp < 18) {
        // ------------------------------------------------------------ diag(u) Z
        for (int c = 0; ok && c < n; ++c) ok = scale_Z(c, (warp - 14) * 32 + lane, 0, 1);
        __syncwarp();
    } else if (warp < 10) {
        // ------------------------------------------------------------ state
        // Lane z, key rows x. Per chunk: the bf16 snapshot of S for X S, and S <- l^n S.
        const int z = j * 32 + lane;
        {
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
            for (int x0 = 0; x0 < Dx; x0 += 64) {       // 64 loads on their way at a time
                uint32_t r[4][16];
#pragma unroll
                for (int x = 0; x < 64; ++x)
                    r[x >> 4][x & 15] = init && z < Dz ? __float_as_uint(init[(x0 + x) * sx + z * sz]) : 0u;
#pragma unroll
                for (int q = 0; q < 4; ++q) tmem_st16(tmem_addr(tm, j, COL_S + x0 + 16 * q), r[q]);
            }
            tmem_wait_st();
        }
        // The state before chunk c (with kExact: after the last one for c = n, which goes to fin).
        for (int c = 0; c < n + (kExact ? 1 : 0); ++c) {
            const bool last = c == n;
            // (U(c - 1) was issued after I(c - 2), so that snapshot's buffer is free, too)
            if (!__all_sync(0xffffffffu, c == 0 || wait_bar(&bars[UDONE], par(c - 1)))) { ok = false; break; }
            tc_fence_after();
            if (!kExact) {
                const float carry = pw[chunk_tokens(cb + c, a)];
                const float2 cc = make_float2(carry, carry);
#pragma unroll 1
                for (int q = 0; q < Dx; q += 32) {
                    float sv[32];
                    tmem_ld32f(tmem_addr(tm, j, COL_S + q), sv);
                    uint32_t pk[16], s0[16], s1[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) pk[x] = pack_bf16(sv[2 * x], sv[2 * x + 1]);
                    tmem_st16(tmem_addr(tm, j, COL_SB + (c & 1) * 64 + q / 2), pk);
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        const float2 lo = mul2(make_float2(sv[x], sv[x + 1]), cc);
                        const float2 hi = mul2(make_float2(sv[16 + x], sv[17 + x]), cc);
                        s0[x] = __float_as_uint(lo.x);
                        s0[x + 1] = __float_as_uint(lo.y);
                        s1[x] = __float_as_uint(hi.x);
                        s1[x + 1] = __float_as_uint(hi.y);
                    }
                    tmem_st16(tmem_addr(tm, j, COL_S + q), s0);
                    tmem_st16(tmem_addr(tm, j, COL_S + q + 16), s1);
                }
            } else {
                // S <- l^n S + D, rounded to nearest (a sum kept in the accumulator over many chunks
                // is cut off at every step: 3e-6 of hT at a memory of 1024 tokens)
                const float carry = c > 0 ? pw[chunk_tokens(cb + c - 1, a)] : 1.f;
                const float2 cc = make_float2(carry, carry);
                float *fp = m.fin + (size_t)bh * Dx * Dz + z;
#pragma unroll 1
                for (int q = 0; q < Dx; q += 32) {
                    uint32_t d0[16], d1[16], s0[16], s1[16];
                    tmem_ld16(tmem_addr(tm, j, COL_S + q), s0);
                    tmem_ld16(tmem_addr(tm, j, COL_S + q + 16), s1);
                    if (c > 0) {
                        tmem_ld16(tmem_addr(tm, j, COL_D + q), d0);
                        tmem_ld16(tmem_addr(tm, j, COL_D + q + 16), d1);
                    }
                    tmem_wait_ld();
                    reg_fence(s0);
                    reg_fence(s1);
                    if (c > 0) {
                        reg_fence(d0);
                        reg_fence(d1);
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            const float2 lo = fma2(make_float2(__uint_as_float(s0[x]), __uint_as_float(s0[x + 1])), cc,
                                                   make_float2(__uint_as_float(d0[x]), __uint_as_float(d0[x + 1])));
                            const float2 hi = fma2(make_float2(__uint_as_float(s1[x]), __uint_as_float(s1[x + 1])), cc,
                                                   make_float2(__uint_as_float(d1[x]), __uint_as_float(d1[x + 1])));
                            s0[x] = __float_as_uint(lo.x);
                            s0[x + 1] = __float_as_uint(lo.y);
                            s1[x] = __float_as_uint(hi.x);
                            s1[x + 1] = __float_as_uint(hi.y);
                        }
                    }
                    if (last) {
                        if (z < Dz) {
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                fp[(q + x) * Dz] = __uint_as_float(s0[x]);
                                fp[(q + 16 + x) * Dz] = __uint_as_float(s1[x]);
                            }
                        }
                        continue;
                    }
                    if (c > 0) {
                        tmem_st16(tmem_addr(tm, j, COL_S + q), s0);
                        tmem_st16(tmem_addr(tm, j, COL_S + q + 16), s1);
                        // the snapshot was last read by I(c - 1)
                        if (q == 0) {
                            if (!__all_sync(0xffffffffu, wait_bar(&bars[SBFREE], par(c - 1)))) ok = false;
                            tc_fence_after();
                        }
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        pk[x] = pack_bf16(__uint_as_float(s0[2 * x]), __uint_as_float(s0[2 * x + 1]));
                        pk[8 + x] = pack_bf16(__uint_as_float(s1[2 * x]), __uint_as_float(s1[2 * x + 1]));
                    }
                    tmem_st16(tmem_addr(tm, j, COL_SB_EXACT + q / 2), pk);
                }
                if (!ok || last) break;
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SREADY]);
        }
        __syncwarp();
    }

    if (!ok) atomicOr(a.err, kDevErrTimeout);
    // launched beside the other maps' kernel: what follows this one must find that complete, too
    if (kExact) pdl_wait_prerequisites();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ======================================================================= state kernel
// Stages of y and z, the latter overwritten with the first part of diag(u) Z. Their number is even:
// each stage then belongs to one of the two groups of scaling warps, which sees every use of it
// (a parity tells a use from the last one, not from the one before).
namespace st {
constexpr uint32_t Y = 0, Z = 16384, STAGE = 32768;
constexpr uint32_t REST = 4 * STAGE;             // the other parts, a buffer for each group
constexpr uint32_t PW = 6 * STAGE;
constexpr uint32_t BAR = PW + 320;
constexpr uint32_t NBAR = 26;
constexpr uint32_t TSLOT = BAR + NBAR * 8;
constexpr uint32_t ALLOC = TSLOT + 16 + 1024;
static_assert(ALLOC <= 232448, "state kernel shared memory");
}  // namespace st
// 0 TMA, 1 MMA, 2-5 and 6-9 diag(u) Z of every other chunk, 10-17 the sum of the accumulators
constexpr int kStateThreads = 576;

struct StateProblem {
    float *E;               // [BH][segs pieces][Dx][Dz]
    float *start;           // [BH][splits - 1][Dx][Dz]
    int li;                 // the map whose y and z it reads
    int segs;               // splits - 1, or splits where the final state is wanted
};
struct StateArgs {
    StateProblem s[2];
    int n, pieces;
    int retain;             // chunks of a CTA (read last) that stay in L2 for the out kernel
};

// Chunks of piece `sub` of segment `seg`, in the order of the walk.
__device__ __forceinline__ void piece_range(const TcArgs &a, int seg, int sub, int pieces, int &cb,
                                            int &ce) {
    const int s0 = seg_bound(seg, a);
    const int len = seg_bound(seg + 1, a) - s0;
    cb = s0 + sub * len / pieces;       // (len < 2^24, pieces <= 8)
    ce = s0 + (sub + 1) * len / pieces;
}

template <int kParts>
__device__ __forceinline__ void state_piece(const TcMaps &maps, const TcArgs &a, const StateArgs &sa,
                                            const StateProblem &sp, int bh, int pi) {
    using namespace st;
    constexpr int NS = 4;
    // Three parts: an accumulator takes kRun chunks, two take turns, and their sums are added in
    // registers (a sum over many chunks in the accumulator would be cut off at each step).
    constexpr int kRun = kParts == 3 ? 2 : 1 << 30;
    enum { SFULL = 0, SEMPTY = NS, SZDONE = 2 * NS, SDONE = 3 * NS, SREAD = SDONE + 2, SZFREE = SREAD + 2,
           SEND = SZFREE + 2 };
    static_assert(SEND < (int)NBAR, "state kernel barrier map");
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = align1024(smraw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + BAR);
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + TSLOT);
    float *pw = reinterpret_cast<float *>(sm + PW);
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int npc = sp.segs * sa.pieces;
    const TcLin &m = a.lin[sp.li];
    const int b = bh / a.H, h = bh % a.H, rev = m.rev, Dx = m.Dx, Dz = m.Dz;
    int cb, ce;
    piece_range(a, pi / sa.pieces, pi % sa.pieces, sa.pieces, cb, ce);
    const int n = ce - cb;
    // the chunks run last to first: what is read last is what the out kernel reads first
    auto start = [&](int c) { return chunk_start(ce - 1 - c, a, rev); };
    const float g = a.decay[h];
    if (threadIdx.x <= kC) pw[threadIdx.x] = decay_pow(g, (float)threadIdx.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&bars[SFULL + i], 1);
            mbar_init(&bars[SEMPTY + i], 1);
            mbar_init(&bars[SZDONE + i], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars[SDONE + i], 1);
            mbar_init(&bars[SREAD + i], 8);
            mbar_init(&bars[SZFREE + i], 1);
        }
        mbar_init(&bars[SEND], 1);
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&maps.y[sp.li]);
        tma_prefetch_desc(&maps.z[sp.li]);
    }
    if (warp == 1) tmem_alloc(tslot, 256);
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
                if (c >= NS && !wait_bar(&bars[SEMPTY + s], par(c / NS - 1))) { ok = false; break; }
                uint8_t *base = sm + s * STAGE;
                const uint64_t pol = c >= n - sa.retain ? keep : drop;
                mbar_arrive_expect_tx(&bars[SFULL + s], (uint32_t)(Dx + Dz) * 2 * kC);
                load_tile(base + Y, &maps.y[sp.li], &bars[SFULL + s], Dx, h / m.hy, start(c), b, pol);
                load_tile(base + Z, &maps.z[sp.li], &bars[SFULL + s], Dz, h / m.hz, start(c), b, pol);
            }
            for (int i = 0; i < NS; ++i) {
                const int uses = c > i ? (c - 1 - i) / NS + 1 : 0;
                if (uses > 0 && !wait_bar(&bars[SFULL + i], par(uses - 1))) ok = false;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idU = idesc_bf16(128, Dx, 1, 1);
        const uint64_t dY = smem_desc(smem_u32(sm) + Y, 8192, 1024);
        const uint64_t dZ = smem_desc(smem_u32(sm) + Z, 8192, 1024);
        const uint64_t dRest = smem_desc(smem_u32(sm) + REST, 8192, 1024);
        for (int c = 0; c < n; ++c) {
            const int run = c / kRun, buf = run & 1;    // (run 0 alone with two parts)
            const bool first = c % kRun == 0, w = wait_bar(&bars[SZDONE + c % NS], par(c / NS)) &&
                               (!first || run < 2 || wait_bar(&bars[SREAD + buf], par((run >> 1) - 1)));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            tc_fence_after();
            const uint64_t so = (uint64_t)((c % NS) * (STAGE >> 4));
            const uint64_t rest = dRest + (uint64_t)((c & 1) * (STAGE >> 4));
            if (elect_one()) {
                // the small parts first
#pragma unroll
                for (int part = kParts - 1; part >= 0; --part)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ss(tm + buf * 128,
                               (part ? rest + (part - 1) * (16384 >> 4) : dZ + so) + kk * (2048 >> 4),
                               dY + so + kk * (2048 >> 4), idU,
                               (!first || part < kParts - 1 || kk > 0) ? 1u : 0u);
                mma_commit(&bars[SEMPTY + c % NS]);
                mma_commit(&bars[SZFREE + (c & 1)]);
                if ((c + 1) % kRun == 0 || c + 1 == n) mma_commit(&bars[SDONE + buf]);
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(&bars[SEND]);
        __syncwarp();
        if (!wait_bar(&bars[SEND], 0)) ok = false;
        __syncwarp();
    } else if (warp < 10) {
        const int ct = ((warp - 2) & 3) * 32 + lane;    // 16-byte vectors ct + 128 x: tokens row + 16 x
        for (int c = (warp - 2) >> 2; c < n; c += 2) {
            const int s = c % NS;
            // tokens that follow this chunk in the piece
            const int p = ce - 1 - c, nt = chunk_tokens(p, a);
            const int rest_tokens = min((int)a.T, ce * kC) - p * kC - nt;
            const float after = m.a_in * decay_pow(g, (float)rest_tokens);
            float u[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) u[x] = after * state_factor(pw, (ct >> 3) + 16 * x, nt, rev);
            const bool w = wait_bar(&bars[SFULL + s], par(c / NS)) &&
                           (c < 2 || wait_bar(&bars[SZFREE + (c & 1)], par((c >> 1) - 1)));
            if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
            uint4 *rest = reinterpret_cast<uint4 *>(sm + REST + (c & 1) * STAGE) + ct;
            uint4 *zs = reinterpret_cast<uint4 *>(sm + s * STAGE + Z) + ct;
#pragma unroll 1
            for (int box = 0; box < Dz / 64; ++box) {
                uint4 v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) v[x] = zs[box * 512 + 128 * x];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    put_scaled<kParts>(v[x], u[x], zs + box * 512 + 128 * x, rest + box * 512 + 128 * x);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SZDONE + s]);
        }
        __syncwarp();
    } else {
        // E^T: lanes z (quarter j), columns x (half) in registers
        const int j = warp & 3, half = (warp - 10) >> 2, z = j * 32 + lane;
        const bool mine = 64 * half < Dx;
        float S[64];
#pragma unroll
        for (int x = 0; x < 64; ++x) S[x] = 0.f;
        const int runs = (n - 1) / kRun + 1;
        for (int r = 0; r < runs; ++r) {
            if (!__all_sync(0xffffffffu, wait_bar(&bars[SDONE + (r & 1)], par(r >> 1)))) { ok = false; break; }
            tc_fence_after();
            if (mine) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float d[32];
                    tmem_ld32f(tmem_addr(tm, j, (r & 1) * 128 + 64 * half + 32 * q), d);
#pragma unroll
                    for (int x = 0; x < 32; ++x) S[32 * q + x] += d[x];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[SREAD + (r & 1)]);
        }
        if (ok && mine && z < Dz) {
            float *ep = sp.E + ((size_t)bh * npc + pi) * (Dx * Dz) + z;
#pragma unroll
            for (int x = 0; x < 64; ++x) ep[(64 * half + x) * Dz] = S[x];
        }
        __syncwarp();
    }
    if (!ok) atomicOr(a.err, kDevErrTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, 256);
    }
}

// CTA = one piece of one problem and head. Measured: 8 of 9 segments of 16 heads of 16384 tokens and
// their final states 35 us (134 MB, 3.8 TB/s: bound by the scaling of Z between the copies and the MMAs).
__global__ void __launch_bounds__(kStateThreads, 1)
hda_tc_state_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a,
                    const __grid_constant__ StateArgs sa) {
    const int n0 = sa.s[0].segs * sa.pieces, all = n0 + (sa.n > 1 ? sa.s[1].segs * sa.pieces : 0);
    const int bh = blockIdx.x / all, i = blockIdx.x % all;
    const StateProblem &sp = sa.s[i < n0 ? 0 : 1];
    const int pi = i < n0 ? i : i - n0;
    if (sp.segs == a.splits) state_piece<3>(maps, a, sa, sp, bh, pi);
    else state_piece<2>(maps, a, sa, sp, bh, pi);
}

// ======================================================================= scan kernel
// Start states of segments 1 .. splits - 1, and the final state. A thread carries kScanPer elements of
// one head; the loads of a batch of pieces are issued together, so the chain costs one round trip
// per batch (16 heads of 8 segments: 8 us from cold caches).
constexpr int kScanThreads = 256, kScanPer = 4, kScanBatch = 12;

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
    const int nseg = a.splits - 1, npc = sp.segs * sa.pieces;
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
            const float f = decay_pow(g, (float)(min((int)a.T, ce * kC) - cb * kC));
            const bool end = (r + 1) % sa.pieces == 0;
            const int seg = r / sa.pieces;
#pragma unroll
            for (int i = 0; i < kScanPer; ++i) {
                s[i] = fmaf(f, s[i], ev[j][i]);
                if (!end) continue;
                if (seg < nseg) ob[(size_t)seg * dd + i * kScanThreads] = s[i];
                else m.fin[bh * dd + e0 + i * kScanThreads] = s[i];
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
    for (const void *k : {(const void *)hda_tc_out_kernel<false>, (const void *)hda_tc_out_kernel<true>}) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, om::ALLOC);
        if (e != cudaSuccess) return e;
    }
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

// The store of a warp's 32 columns of a contiguous [B, T, H, D] output: 64 tokens of bf16 (rows of 64
// bytes, swizzled), or 32 of float.
bool make_out_map(CUtensorMap *m, void *out, bool f32, int64_t B, int64_t T, int64_t H, int64_t D) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    const cuuint64_t es = f32 ? 4 : 2;
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t strides[3] = {D * es, H * D * es, T * H * D * es};
    cuuint32_t box[4] = {32, 1, f32 ? 32u : kC, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, out, dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              f32 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_64B,
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
// `segs`: segments of all problems together.
int state_pieces(const HdaProblem &p, int splits, int segs, int sms) {
    if (splits <= 1) return 1;
    const int64_t nchunks = (p.T + kC - 1) / kC;
    int64_t k = sms / (p.B * p.H * segs);
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
        if (p.T * p.H * m.Dz * 4 >= (int64_t(1) << 40)) return false;
    }
    return true;
}

size_t hda_tc_workspace_bytes(const HdaProblem &p, int splits, int num_sms) {
    const int s = clamp_splits(p, splits, num_sms);
    if (s <= 1) return 0;
    // E of every piece (one segment more where the final state is wanted: room for it always, since
    // the size must not depend on it) and the start states
    const size_t per = (size_t)(p.B * p.H) * p.lin[0].Dx * p.lin[0].Dz * sizeof(float);
    const int pieces = state_pieces(p, s, state_problems(p) * (s - 1), num_sms);
    return state_problems(p) * per * ((size_t)s * pieces + (s - 1));
}

cudaError_t launch_hda_tc(const HdaProblem &p, int splits, int num_sms, void *ws,
                          unsigned int *dev_err, cudaStream_t stream) {
    cudaError_t e = set_attrs();
    if (e != cudaSuccess) return e;
    const int s = clamp_splits(p, splits, num_sms), ns = state_problems(p);
    int segs = 0;
    for (int i = 0; i < ns; ++i) segs += p.lin[2 * i].fin ? s : s - 1;
    const int pieces = state_pieces(p, s, segs, num_sms);
    const int64_t bh = p.B * p.H;
    TcMaps maps{};
    TcArgs a{};
    a.decay = p.decay;
    a.T = p.T;
    a.n = p.n;
    a.H = (int)p.H;
    a.nchunks = (int)((p.T + kC - 1) / kC);
    a.splits = s;
    a.seg_len = a.nchunks / s;
    a.seg_more = a.nchunks % s;
    a.hint = p.n == 1;
    a.err = dev_err;
    for (int i = 0; i < p.n; ++i) {
        const HdaLin &m = p.lin[i];
        if (!make_map(&maps.x[i], m.x, p.B, p.T, m.Dx) || !make_map(&maps.y[i], m.y, p.B, p.T, m.Dx) ||
            !make_map(&maps.z[i], m.z, p.B, p.T, m.Dz) ||
            !make_out_map(&maps.o[i], m.out, m.out_f32, p.B, p.T, p.H, m.Dz))
            return cudaErrorInvalidResourceHandle;   // a tensor map could not be encoded
        const auto rep = [&](const HdaTensor &t) { return (int)(p.H / t.heads); };
        a.lin[i] = TcLin{m.init, nullptr, m.fin, m.out, m.init_t, 0, m.out_f32, m.Dx, m.Dz,
                         rep(m.x), rep(m.y), rep(m.z), m.a_in, m.a_out, m.rev};
    }
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    if (s > 1) {
        const size_t per = (size_t)bh * p.lin[0].Dx * p.lin[0].Dz;
        StateArgs sa{};
        sa.n = ns;
        sa.pieces = pieces;
        float *w = static_cast<float *>(ws);
        const int64_t all = (int64_t)segs * pieces;
        for (int i = 0; i < ns; ++i) {
            StateProblem &sp = sa.s[i];
            sp.li = 2 * i;
            sp.segs = p.lin[2 * i].fin ? s : s - 1;
            sp.E = w;
            sp.start = w + per * s * pieces;
            w += per * (s * pieces + s - 1);
            a.lin[2 * i].start = sp.start;
        }
        if (p.n == 3) {
            a.lin[1].start = a.lin[2].start;
            a.lin[1].start_t = 1;
        }
        // keep about kL2Keep bytes of what the state pass reads last for the out kernel
        sa.retain = (int)std::min<int64_t>((a.nchunks / s + pieces - 1) / pieces,
                                           kL2Keep / (bh * all * (p.lin[0].Dx + p.lin[0].Dz) * kC * 2));
        hda_tc_state_kernel<<<(unsigned)(bh * all), kStateThreads, st::ALLOC, stream>>>(maps, a, sa);
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
    // the last map may return a state: if nothing is split, from the output kernel
    const int exact = s == 1 && p.lin[p.n - 1].fin ? 1 : 0, plain = p.n - exact;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kOutThreads);
    cfg.dynamicSmemBytes = om::ALLOC;
    cfg.stream = stream;
    cfg.attrs = pdl;
    if (plain > 0) {
        cfg.gridDim = dim3((unsigned)(bh * s * plain));
        cfg.numAttrs = s > 1 ? 1 : 0;
        if ((e = cudaLaunchKernelEx(&cfg, hda_tc_out_kernel<false>, maps, a, 0, plain)) != cudaSuccess) return e;
        count_launches(1);
    }
    if (exact > 0) {
        // depends on nothing the other kernel writes: its CTAs fill the SMs as that one's end
        cfg.gridDim = dim3((unsigned)(bh * s));
        cfg.numAttrs = plain > 0 ? 1 : 0;
        if ((e = cudaLaunchKernelEx(&cfg, hda_tc_out_kernel<true>, maps, a, plain, 1)) != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace gla
