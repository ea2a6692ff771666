// Pages of a pool of recurrent states: copied, forked, freed and compacted on the device.
//
// A request list is planned by one CTA (who gets which page: prefix sums over the requests in
// their order, so the result is that of a sequential walk), which writes the list of moves; a
// second kernel, launched as its programmatic dependent, carries the pages over. Planning reads
// a few integers per page and is bound by latency; the copy by HBM bandwidth. Measured: 64 pages of
// 1 MB forked 7.5 + 17.6 us, 640 pages of 256 KB compacted 7.2 + 14 us.
#include "gla_internal.h"
#include "pages.h"
#include "tc_ptx.cuh"

namespace gla {
namespace {

constexpr int kPlan = 1024;                 // threads of a planning CTA
constexpr int kNone = 0x7fffffff;
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;                // 16-byte vectors a thread moves per unit
constexpr int64_t kUnit = (int64_t)kCopyThreads * kCopyVecs * 16;   // bytes

struct Move {
    int src, dst;
};

// Exclusive prefix of v over the planning CTA in thread order; `total` is the sum.
__device__ __forceinline__ int block_prefix(int v, int *sh, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int w = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return x - v + (warp > 0 ? before : 0);
}

// Pages on the stack as the count says, held to [0, P].
__device__ __forceinline__ int stack_count(const PagePool &p, unsigned *err) {
    const int c = *p.count;
    if (c >= 0 && c <= p.P) return c;
    if (threadIdx.x == 0) atomicOr(err, kDevErrPages);
    return c < 0 ? 0 : (int)p.P;
}

// Workspace of a fork: n_moves, first [R] (the first request that names a row as its child),
// use [n] (1: the request is carried out), moves [n * M].
__global__ void __launch_bounds__(kPlan)
pages_fork_plan(const PagePool p, const int *__restrict__ parents, const int *__restrict__ children,
                int n, int *n_moves, int *first, int *use, Move *moves, unsigned *err) {
    tc::pdl_launch_dependents();
    __shared__ int sh[32];
    const int R = (int)p.R, M = (int)p.M;
    for (int r = threadIdx.x; r < R; r += kPlan) first[r] = kNone;
    const int have = stack_count(p, err);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int a = parents[i], c = children[i];
        if (a >= 0 && c >= 0 && a < R && c < R) atomicMin(&first[c], i);
    }
    __syncthreads();
    // Whether a request is carried out, from the table as it is before the call. A parent that
    // has no pages gives none; one that has pages cannot be a child, so no row is both read
    // and written below.
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int a = parents[i], c = children[i];
        bool ok = a >= 0 && c >= 0;
        if (ok) {
            bool bad = a >= R || c >= R;
            if (!bad) {
                bad = first[c] != i;
                for (int m = 0; m < M; ++m) bad |= p.table[(int64_t)c * M + m] >= 0;
            }
            if (bad) {
                atomicOr(err, kDevErrPages);
                ok = false;
            } else {
                ok = false;
                for (int m = 0; m < M; ++m) ok |= p.table[(int64_t)a * M + m] >= 0;
            }
        }
        use[i] = ok;
    }
    __syncthreads();
    int done = 0, moved = 0;   // entries that want a page so far, moves so far
    for (int64_t e0 = 0; e0 < (int64_t)n * M; e0 += kPlan) {
        const int64_t e = e0 + threadIdx.x;
        int src = -1, c = -1, m = 0;
        if (e < (int64_t)n * M) {
            const int i = (int)(e / M);
            m = (int)(e % M);
            if (use[i]) {
                c = children[i];
                src = p.table[(int64_t)parents[i] * M + m];
                if (src >= p.P) {
                    atomicOr(err, kDevErrPages);
                    src = -1;
                }
            }
        }
        int total;
        const int rank = done + block_prefix(src >= 0, sh, total);
        int dst = -1;
        if (src >= 0) {
            if (rank < have) dst = p.free_stack[have - 1 - rank];
            if (dst < 0 || dst >= p.P) {
                atomicOr(err, kDevErrPages);
                dst = -1;
            }
        }
        int made;
        const int at = moved + block_prefix(dst >= 0, sh, made);
        if (c >= 0) p.table[(int64_t)c * M + m] = dst;
        if (dst >= 0) moves[at] = Move{src, dst};
        done += total;
        moved += made;
    }
    if (threadIdx.x == 0) {
        *n_moves = moved;
        *p.count = have - min(done, have);
    }
}

__global__ void __launch_bounds__(kPlan)
pages_free_plan(const PagePool p, const int *__restrict__ rows, int n, int *first, unsigned *err) {
    __shared__ int sh[32];
    const int R = (int)p.R, M = (int)p.M;
    for (int r = threadIdx.x; r < R; r += kPlan) first[r] = kNone;
    const int have = stack_count(p, err);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kPlan) {
        const int r = rows[i];
        if (r >= 0 && r < R) atomicMin(&first[r], i);
        else if (r >= R) atomicOr(err, kDevErrPages);
    }
    __syncthreads();
    // pass 0 counts the pages; pass 1 pushes them, the last of the list first
    int all = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int done = 0;
        for (int64_t e0 = 0; e0 < (int64_t)n * M; e0 += kPlan) {
            const int64_t e = e0 + threadIdx.x;
            int page = -1;
            int64_t at = -1;
            if (e < (int64_t)n * M) {
                const int i = (int)(e / M), r = rows[i];
                if (r >= 0 && r < R && first[r] == i) {
                    at = (int64_t)r * M + e % M;
                    page = p.table[at];
                    if (page >= p.P) {
                        atomicOr(err, kDevErrPages);
                        page = -1;
                    }
                }
            }
            int total;
            const int rank = done + block_prefix(page >= 0, sh, total);
            if (pass == 1) {
                if (page >= 0) {
                    const int to = have + all - 1 - rank;
                    if (to < p.P) p.free_stack[to] = page;
                    else atomicOr(err, kDevErrPages);   // more pages than the pool has
                }
                if (at >= 0) p.table[at] = -1;
            }
            done += total;
        }
        all = done;
    }
    if (threadIdx.x == 0) *p.count = min(have + all, (int)p.P);
}

// Workspace of a compaction: n_moves, map [P] (first whether a page is live, then where it
// goes), holes [P], moves [P].
__global__ void __launch_bounds__(kPlan)
pages_compact_plan(const PagePool p, int *n_moves, int *map, int *holes, Move *moves,
                   unsigned *err) {
    tc::pdl_launch_dependents();
    __shared__ int sh[32];
    const int P = (int)p.P;
    const int64_t entries = p.R * p.M;
    for (int i = threadIdx.x; i < P; i += kPlan) map[i] = 0;
    __syncthreads();
    for (int64_t e = threadIdx.x; e < entries; e += kPlan) {
        const int page = p.table[e];
        if (page >= P || (page >= 0 && atomicExch(&map[page], 1) != 0)) atomicOr(err, kDevErrPages);
    }
    __syncthreads();
    int live = 0;
    for (int i0 = 0; i0 < P; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        int total;
        block_prefix(i < P && map[i], sh, total);
        live += total;
    }
    int nh = 0, nm = 0;
    for (int i0 = 0; i0 < P; i0 += kPlan) {
        const int i = i0 + threadIdx.x;
        const bool is = i < P && map[i] != 0, hole = i < live && !is, up = is && i >= live;
        int th, tm;
        const int rh = nh + block_prefix(hole, sh, th);
        const int rm = nm + block_prefix(up, sh, tm);
        if (hole) holes[rh] = i;
        if (up) moves[rm].src = i;
        nh += th;
        nm += tm;
    }
    __syncthreads();
    // as many live pages lie at or above the live count as there are holes below it
    for (int i = threadIdx.x; i < P; i += kPlan) {
        map[i] = i;
        p.free_stack[i] = i < P - live ? P - 1 - i : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nm; i += kPlan) {
        moves[i].dst = holes[i];
        map[moves[i].src] = holes[i];
    }
    __syncthreads();
    for (int64_t e = threadIdx.x; e < entries; e += kPlan) {
        const int page = p.table[e];
        if (page >= 0 && page < P) p.table[e] = map[page];
        else if (page < 0) p.table[e] = -1;
    }
    if (threadIdx.x == 0) {
        *n_moves = nm;
        *p.count = P - live;
    }
}

// Page src -> page dst for every move; the moves come from the plan (count on the device), or
// from the caller's two lists (checked here).
__global__ void __launch_bounds__(kCopyThreads)
pages_move_kernel(char *pool, int64_t P, int64_t page_bytes, const int *n_moves, const Move *moves,
                  const int *src, const int *dst, int64_t n, unsigned *err) {
    tc::pdl_wait_prerequisites();
    if (n_moves) n = *n_moves;
    const int64_t per = (page_bytes + kUnit - 1) / kUnit, units = n * per;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / per, off = u % per * kUnit;
        const int64_t a = moves ? moves[i].src : src[i], b = moves ? moves[i].dst : dst[i];
        if (a < 0 || b < 0 || a == b) continue;
        if (a >= P || b >= P) {
            if (off == 0 && threadIdx.x == 0) atomicOr(err, kDevErrPages);
            continue;
        }
        const uint4 *s = reinterpret_cast<const uint4 *>(pool + a * page_bytes + off);
        uint4 *d = reinterpret_cast<uint4 *>(pool + b * page_bytes + off);
        const int64_t left = (page_bytes - off) / 16;
        uint4 v[kCopyVecs];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j) {
            const int k = threadIdx.x + j * kCopyThreads;
            if (k < left) v[j] = s[k];
        }
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j) {
            const int k = threadIdx.x + j * kCopyThreads;
            if (k < left) d[k] = v[j];
        }
    }
}

// `most`: moves at most (the grid need not hold them all).
cudaError_t launch_moves(const PagePool &p, const int *n_moves, const Move *moves, const int *src,
                         const int *dst, int64_t n, int64_t most, int num_sms, unsigned *err,
                         bool dependent, cudaStream_t s) {
    const int64_t per = (p.page_bytes + kUnit - 1) / kUnit;
    if (most * per == 0) return cudaSuccess;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)min(most * per, (int64_t)num_sms * 8));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = dependent ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, pages_move_kernel, static_cast<char *>(p.pool), p.P,
                                             p.page_bytes, n_moves, moves, src, dst, n, err);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace

size_t pages_fork_workspace(const PagePool &p, int64_t n) {
    return (size_t)(2 + p.R + n + 2 * n * p.M + 2) * 4;
}
size_t pages_free_workspace(const PagePool &p) { return (size_t)(p.R > 4 ? p.R : 4) * 4; }
size_t pages_compact_workspace(const PagePool &p) { return (size_t)(2 + 4 * p.P) * 4; }

cudaError_t launch_pages_copy(const PagePool &p, const int *src, const int *dst, int64_t n,
                              int num_sms, unsigned int *dev_err, cudaStream_t s) {
    return launch_moves(p, nullptr, nullptr, src, dst, n, n, num_sms, dev_err, false, s);
}

cudaError_t launch_pages_fork(const PagePool &p, const int *parents, const int *children, int64_t n,
                              void *ws, int num_sms, unsigned int *dev_err, cudaStream_t s) {
    int *w = static_cast<int *>(ws);
    Move *moves = reinterpret_cast<Move *>(w + 2);
    int *first = w + 2 + 2 * n * p.M, *use = first + p.R;
    pages_fork_plan<<<1, kPlan, 0, s>>>(p, parents, children, (int)n, w, first, use, moves, dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    return launch_moves(p, w, moves, nullptr, nullptr, 0, n * p.M, num_sms, dev_err, true, s);
}

cudaError_t launch_pages_free(const PagePool &p, const int *rows, int64_t n, void *ws,
                              unsigned int *dev_err, cudaStream_t s) {
    pages_free_plan<<<1, kPlan, 0, s>>>(p, rows, (int)n, static_cast<int *>(ws), dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t launch_pages_compact(const PagePool &p, void *ws, int num_sms, unsigned int *dev_err,
                                 cudaStream_t s) {
    int *w = static_cast<int *>(ws);
    Move *moves = reinterpret_cast<Move *>(w + 2);
    int *map = w + 2 + 2 * p.P, *holes = map + p.P;
    pages_compact_plan<<<1, kPlan, 0, s>>>(p, w, map, holes, moves, dev_err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    count_launches(1);
    // no more pages move than half the pool, and none than the table has entries
    const int64_t most = min(p.P / 2 + 1, p.R * p.M);
    return launch_moves(p, w, moves, nullptr, nullptr, 0, most, num_sms, dev_err, true, s);
}

}  // namespace gla
