// C ABI of the decay attention (hda_*), the group norm (gla_group_norm_*) and the state pages
// (gla_pages_*): argument checks, path choice, workspace. See include/gla.h for the contracts.
#include <algorithm>
#include <stdio.h>

#include "gla.h"
#include "gla_internal.h"
#include "hda_internal.h"
#include "norm.h"
#include "pages.h"

namespace {

constexpr int64_t kMostElems = int64_t(1) << 62;

bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

// a * b of non-negative sizes; false past 2^62 (so byte counts still fit)
bool mul_ok(int64_t a, int64_t b, int64_t *r) {
    if (a < 0 || b < 0 || (a != 0 && b > kMostElems / 16 / a)) return false;
    *r = a * b;
    return true;
}

// A memory range an argument covers.
struct Range {
    const void *p;
    int64_t bytes;
};
bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (size_t)b.bytes && y < x + (size_t)a.bytes;
}
// GLA_ERR_ALIAS if an output overlaps an input or another output.
gla_status check_alias(const Range *outs, int no, const Range *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int j = 0; j < ni; ++j)
            if (overlap(outs[i], ins[j])) return GLA_ERR_ALIAS;
        for (int j = i + 1; j < no; ++j)
            if (overlap(outs[i], outs[j])) return GLA_ERR_ALIAS;
    }
    return GLA_OK;
}

// The caller's workspace if it will do, else the stream's own.
gla_status get_workspace(void *ws, size_t bytes, size_t need, cudaStream_t s, const Range *used,
                         int nu, void **out) {
    *out = nullptr;
    if (ws) {
        if (misaligned(ws) || bytes < need) return GLA_ERR_WORKSPACE;
        for (int i = 0; i < nu; ++i)
            if (overlap(Range{ws, (int64_t)need}, used[i])) return GLA_ERR_WORKSPACE;
        *out = ws;
        return GLA_OK;
    }
    if (need == 0) return GLA_OK;
    return (gla_status)gla::stream_workspace(s, need, out);
}

// Strides of a [b, t, h, D] tensor (contiguous where the caller's are all zero) and its extent
// in bytes. Dimensions of one element take the stride they would have in a packed tensor,
// whatever the caller's says.
gla_status strides_of(const gla_strides &in, int64_t B, int64_t T, int64_t heads, int64_t D, int es,
                      gla::HdaTensor *t, int64_t *bytes) {
    int64_t n;
    if (!mul_ok(heads, D, &n) || !mul_ok(n, T, &n) || !mul_ok(n, B, &n)) return GLA_ERR_BAD_SHAPE;
    t->heads = (int)heads;
    if (in.b == 0 && in.t == 0 && in.h == 0) {
        t->h = D;
        t->t = heads * D;
        t->b = T * heads * D;
    } else {
        t->h = heads > 1 ? in.h : D;
        t->t = T > 1 ? in.t : heads * D;
        t->b = B > 1 ? in.b : std::max<int64_t>(T, 1) * heads * D;
        for (int64_t s : {t->h, t->t, t->b})
            if (s <= 0 || (s * es) % 16 != 0) return GLA_ERR_MISALIGNED;
    }
    if (n == 0) {
        *bytes = 0;
        return GLA_OK;
    }
    int64_t last = D, part;
    if (!mul_ok(B - 1, t->b, &part) || (last += part) < 0) return GLA_ERR_BAD_SHAPE;
    if (!mul_ok(T - 1, t->t, &part) || (last += part) < 0) return GLA_ERR_BAD_SHAPE;
    if (!mul_ok(heads - 1, t->h, &part) || (last += part) < 0) return GLA_ERR_BAD_SHAPE;
    if (last > kMostElems / 16) return GLA_ERR_BAD_SHAPE;
    *bytes = last * es;
    return GLA_OK;
}

struct HdaDims {
    int es;
    gla::HdaTensor q, k, v, go;
    int64_t bq, bk, bv, bgo, bo, bs;   // bytes each argument covers
};

gla_status hda_dims(const hda_shape *sh, bool step, HdaDims *d) {
    if (!sh) return GLA_ERR_NULL_ARG;
    if (sh->io != GLA_IO_BF16 && sh->io != GLA_IO_F32) return GLA_ERR_BAD_OPTION;
    const int64_t T = step ? 1 : sh->T;
    if (sh->B < 0 || T < 0 || sh->H < 0) return GLA_ERR_BAD_SHAPE;
    for (int64_t h : {sh->Hq, sh->Hk, sh->Hv})
        if (sh->H > 0 ? (h <= 0 || sh->H % h != 0) : h != 0) return GLA_ERR_BAD_SHAPE;
    if (step) {
        if (sh->Dk < 1 || sh->Dk > 1024 || sh->Dv < 4 || sh->Dv > 1024 || sh->Dv % 4 != 0)
            return GLA_ERR_UNSUPPORTED_DIM;
    } else {
        for (int64_t n : {sh->Dk, sh->Dv})
            if (n < 8 || n > 256 || n % 8 != 0) return GLA_ERR_UNSUPPORTED_DIM;
    }
    int64_t bh, n;
    if (!mul_ok(sh->B, sh->H, &bh) || bh > (int64_t(1) << 30) || T > (int64_t(1) << 30))
        return GLA_ERR_BAD_SHAPE;
    d->es = sh->io == GLA_IO_BF16 ? 2 : 4;
    gla_strides q = sh->q, k = sh->k, v = sh->v;
    if (step) {   // one token: the t strides say nothing; rows need no 16-byte alignment
        int64_t bytes;
        auto one = [&](gla_strides &s, int64_t heads, int64_t D, gla::HdaTensor *t, int64_t *out) {
            t->heads = (int)heads;
            t->t = 0;
            t->h = heads > 1 && (s.b || s.h) ? s.h : D;
            t->b = sh->B > 1 && (s.b || s.h) ? s.b : heads * D;
            if (t->h <= 0 || t->b <= 0) return sh->B * heads == 0;
            int64_t a, c;
            if (!mul_ok(std::max<int64_t>(sh->B - 1, 0), t->b, &a) ||
                !mul_ok(std::max<int64_t>(heads - 1, 0), t->h, &c))
                return false;
            bytes = (a + c + D) * d->es;
            *out = sh->B * heads == 0 ? 0 : bytes;
            return true;
        };
        d->bq = d->bk = d->bv = 0;
        if (!one(q, sh->Hq, sh->Dk, &d->q, &d->bq) || !one(k, sh->Hk, sh->Dk, &d->k, &d->bk) ||
            !one(v, sh->Hv, sh->Dv, &d->v, &d->bv))
            return GLA_ERR_BAD_SHAPE;
    } else {
        gla_status rc = strides_of(q, sh->B, T, sh->Hq, sh->Dk, d->es, &d->q, &d->bq);
        if (rc == GLA_OK) rc = strides_of(k, sh->B, T, sh->Hk, sh->Dk, d->es, &d->k, &d->bk);
        if (rc == GLA_OK) rc = strides_of(v, sh->B, T, sh->Hv, sh->Dv, d->es, &d->v, &d->bv);
        if (rc == GLA_OK) rc = strides_of(sh->d_o, sh->B, T, sh->H, sh->Dv, d->es, &d->go, &d->bgo);
        if (rc != GLA_OK) return rc;
    }
    if (!mul_ok(bh, T, &n) || !mul_ok(n, sh->Dv, &n)) return GLA_ERR_BAD_SHAPE;
    d->bo = n * d->es;
    if (!mul_ok(bh, sh->Dk * sh->Dv, &n)) return GLA_ERR_BAD_SHAPE;
    d->bs = n * 4;
    return GLA_OK;
}

gla_status check_options(const gla_options *opt) {
    if (!opt) return GLA_OK;
    if (opt->path < GLA_PATH_AUTO || opt->path > GLA_PATH_TC || opt->seq_splits < 0 ||
        opt->gate != GLA_GATE_KEY)
        return GLA_ERR_BAD_OPTION;
    return GLA_OK;
}

// GLA_PATH_EXACT / GLA_PATH_TC, or -1.
int hda_path(const gla::HdaProblem &p, const gla_options *opt) {
    const int want = opt ? opt->path : GLA_PATH_AUTO;
    const bool tc = gla::hda_tc_supported(p);
    if (want == GLA_PATH_TC) return tc ? GLA_PATH_TC : -1;
    if (want == GLA_PATH_EXACT) return GLA_PATH_EXACT;
    // a sequence shorter than one chunk is a few tokens' walk for the exact kernel
    return tc && p.T >= 64 ? GLA_PATH_TC : GLA_PATH_EXACT;
}

// The maps of the forward (or, with d_o, of the gradients) without their pointers' checks.
gla::HdaProblem hda_problem(const hda_shape &sh, const HdaDims &d, bool backward, float scale) {
    gla::HdaProblem p{};
    p.B = sh.B;
    p.T = sh.T;
    p.H = sh.H;
    p.io = sh.io;
    const int Dk = (int)sh.Dk, Dv = (int)sh.Dv;
    auto lin = [&](int i, const gla::HdaTensor &x, const gla::HdaTensor &y, const gla::HdaTensor &z,
                   int Dx, int Dz, float a_in, float a_out, int rev) {
        gla::HdaLin &m = p.lin[i];
        m.x = x;
        m.y = y;
        m.z = z;
        m.Dx = Dx;
        m.Dz = Dz;
        m.a_in = a_in;
        m.a_out = a_out;
        m.rev = rev;
    };
    if (!backward) {
        p.n = 1;
        lin(0, d.q, d.k, d.v, Dk, Dv, 1.f, scale, 0);
    } else {
        p.n = 3;
        lin(0, d.go, d.v, d.k, Dv, Dk, 1.f, scale, 0);
        lin(1, d.v, d.go, d.q, Dv, Dk, scale, 1.f, 1);
        lin(2, d.k, d.q, d.go, Dk, Dv, scale, 1.f, 1);
    }
    return p;
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace of a call: the segments' states of either path, then one fp32 buffer per gradient of a
// shared head ([B, T, H, D]).
size_t hda_workspace(const hda_shape &sh, const gla::HdaProblem &p, const gla_options *opt,
                     int path, int sms, size_t *state_bytes) {
    const int splits = opt ? opt->seq_splits : 0;
    size_t need = round256(path == GLA_PATH_TC ? gla::hda_tc_workspace_bytes(p, splits, sms)
                                               : gla::hda_exact_workspace_bytes(p, splits, sms));
    *state_bytes = need;
    if (p.n == 3) {
        const int64_t heads[3] = {sh.Hq, sh.Hk, sh.Hv};
        for (int i = 0; i < 3; ++i)
            if (heads[i] != sh.H) need += round256((size_t)(sh.B * sh.T * sh.H * p.lin[i].Dz) * 4);
    }
    return need;
}

size_t workspace_size(const hda_shape *sh, const gla_options *opt, bool backward) {
    HdaDims d;
    if (hda_dims(sh, false, &d) != GLA_OK || check_options(opt) != GLA_OK) return 0;
    if (sh->B * sh->H * sh->T == 0) return 0;
    const gla::HdaProblem p = hda_problem(*sh, d, backward, 1.f);
    const int path = hda_path(p, opt);
    if (path < 0) return 0;
    int sms;
    unsigned *err;
    gla::device_info(&sms, &err);
    size_t states;
    return hda_workspace(*sh, p, opt, path, sms, &states);
}

// State at the end of no tokens: the one at the start, or zero.
gla_status empty_state(float *dst, const float *src, int64_t bytes, cudaStream_t s) {
    if (!dst || bytes == 0) return GLA_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                              : cudaMemsetAsync(dst, 0, bytes, s);
    return e == cudaSuccess ? GLA_OK
                            : (gla_status)gla::launch_failed("state of an empty sequence", e);
}

gla_status run_hda(gla::HdaProblem &p, const hda_shape &sh, const gla_options *opt, void *ws,
                   size_t state_bytes, int path, int sms, unsigned *err, cudaStream_t s) {
    // gradients of shared heads go to fp32 buffers first
    gla::HdaShare parts[3];
    int np = 0;
    char *at = static_cast<char *>(ws) + state_bytes;
    if (p.n == 3) {
        const int64_t heads[3] = {sh.Hq, sh.Hk, sh.Hv};
        for (int i = 0; i < 3; ++i) {
            if (heads[i] == sh.H) continue;
            gla::HdaLin &m = p.lin[i];
            parts[np++] = gla::HdaShare{reinterpret_cast<float *>(at), m.out, (int)heads[i], m.Dz};
            m.out = at;
            m.out_f32 = 1;
            at += round256((size_t)(sh.B * sh.T * sh.H * m.Dz) * 4);
        }
    }
    cudaError_t e = path == GLA_PATH_TC
                        ? gla::launch_hda_tc(p, opt ? opt->seq_splits : 0, sms, ws, err, s)
                        : gla::launch_hda_exact(p, opt ? opt->seq_splits : 0, sms, ws, s);
    if (e == cudaSuccess) e = gla::launch_hda_share(parts, np, sh.B * sh.T, sh.H, sh.io, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("decay attention launch", e);
}

gla_status norm_problem(const gla_norm_shape *sh, gla::NormProblem *p, int64_t *bx, int64_t *bg,
                        int64_t *bdy, int64_t *by) {
    if (!sh) return GLA_ERR_NULL_ARG;
    if (sh->io != GLA_IO_BF16 && sh->io != GLA_IO_F32) return GLA_ERR_BAD_OPTION;
    if (sh->act < GLA_ACT_NONE || sh->act > GLA_ACT_GELU) return GLA_ERR_BAD_OPTION;
    if (sh->N < 0 || sh->L < 0 || sh->C < 0) return GLA_ERR_BAD_SHAPE;
    if (sh->G <= 0 || sh->C % sh->G != 0) return GLA_ERR_BAD_SHAPE;
    if (!(sh->eps >= 0.f)) return GLA_ERR_BAD_OPTION;
    int64_t n, ng;
    if (!mul_ok(sh->N, sh->L, &n) || !mul_ok(n, sh->C, &n) || !mul_ok(sh->N, sh->G, &ng) ||
        ng > (int64_t(1) << 31) - 1 || sh->C > (int64_t(1) << 24) || sh->L > (int64_t(1) << 31) - 1)
        return GLA_ERR_BAD_SHAPE;
    const int es = sh->io == GLA_IO_BF16 ? 2 : 4;
    *by = n * es;
    *p = gla::NormProblem{};
    p->N = sh->N;
    p->L = sh->L;
    p->C = sh->C;
    p->G = sh->G;
    p->eps = sh->eps;
    p->act = sh->act;
    p->io = sh->io;
    auto one = [&](int64_t sn, int64_t sl, int64_t *pn, int64_t *pl, int64_t *bytes) {
        if (sn == 0 && sl == 0) {
            sl = sh->C;
            sn = sh->L * sh->C;
        }
        *pn = sh->N > 1 ? sn : sh->L * sh->C;
        *pl = sh->L > 1 ? sl : sh->C;
        *bytes = 0;
        if (n == 0) return true;
        if (*pn <= 0 || *pl <= 0) return false;
        int64_t a, b;
        if (!mul_ok(sh->N - 1, *pn, &a) || !mul_ok(sh->L - 1, *pl, &b)) return false;
        *bytes = (a + b + sh->C) * es;
        return true;
    };
    if (!one(sh->x_n, sh->x_l, &p->x_n, &p->x_l, bx) ||
        !one(sh->gate_n, sh->gate_l, &p->gate_n, &p->gate_l, bg) ||
        !one(sh->dy_n, sh->dy_l, &p->dy_n, &p->dy_l, bdy))
        return GLA_ERR_BAD_SHAPE;
    return GLA_OK;
}

// Element alignment of a strided tensor's base (rows may start anywhere).
bool unaligned(const void *p, int io) {
    return p && (reinterpret_cast<uintptr_t>(p) & (io == GLA_IO_BF16 ? 1u : 3u));
}

gla_status check_pool(void *pool, int64_t P, int64_t page_bytes) {
    int64_t n;
    if (P < 0 || P > (int64_t(1) << 30) || page_bytes < 0 || !mul_ok(P, page_bytes, &n))
        return GLA_ERR_BAD_SHAPE;
    if (page_bytes % 16 != 0 || misaligned(pool)) return GLA_ERR_MISALIGNED;
    if (n > 0 && !pool) return GLA_ERR_NULL_ARG;
    return GLA_OK;
}
bool bad_int(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u); }

gla_status check_table(int64_t P, const int32_t *table, int64_t R, int64_t M, const int32_t *stack,
                       const int32_t *count, int64_t n) {
    int64_t e;
    if (P < 0 || P > (int64_t(1) << 30) || R < 0 || M < 0 || n < 0 || n > (int64_t(1) << 30) ||
        R > (int64_t(1) << 30) || M > (int64_t(1) << 30) || !mul_ok(R, M, &e) ||
        e > (int64_t(1) << 30) || !mul_ok(n, M, &e) || e > (int64_t(1) << 30))
        return GLA_ERR_BAD_SHAPE;
    if ((R * M > 0 && !table) || (P > 0 && !stack) || !count) return GLA_ERR_NULL_ARG;
    if (bad_int(table) || bad_int(stack) || bad_int(count)) return GLA_ERR_MISALIGNED;
    return GLA_OK;
}

}  // namespace

extern "C" {

int hda_path_for(const hda_shape *shape, const gla_options *opt) {
    HdaDims d;
    if (hda_dims(shape, false, &d) != GLA_OK || check_options(opt) != GLA_OK) return -1;
    return hda_path(hda_problem(*shape, d, false, 1.f), opt);
}

size_t hda_fwd_workspace_size(const hda_shape *shape, const gla_options *opt) {
    return workspace_size(shape, opt, false);
}
size_t hda_bwd_workspace_size(const hda_shape *shape, const gla_options *opt) {
    return workspace_size(shape, opt, true);
}

gla_status hda_fwd(const void *q, const void *k, const void *v, const float *decay, float scale,
                   const float *h0, void *o, float *hT, const hda_shape *shape,
                   const gla_options *opt, gla_stream_t stream) {
    HdaDims d;
    gla_status rc = hda_dims(shape, false, &d);
    if (rc == GLA_OK) rc = check_options(opt);
    if (rc != GLA_OK) return rc;
    const hda_shape &sh = *shape;
    const bool none = sh.B * sh.H == 0, empty = none || sh.T == 0;
    if (!empty && (!q || !k || !v || !decay || !o)) return GLA_ERR_NULL_ARG;
    for (const void *p : {q, k, v, (const void *)h0, (const void *)o, (const void *)hT})
        if (misaligned(p)) return GLA_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(decay) & 3u) return GLA_ERR_MISALIGNED;
    const Range used[7] = {{q, d.bq}, {k, d.bk}, {v, d.bv}, {decay, sh.H * 4}, {h0, d.bs},
                           {o, d.bo}, {hT, d.bs}};
    if ((rc = check_alias(used + 5, 2, used, 5)) != GLA_OK) return rc;
    gla::HdaProblem p = hda_problem(sh, d, false, scale);
    const int path = hda_path(p, opt);
    if (path < 0) return GLA_ERR_UNSUPPORTED_DIM;
    p.decay = decay;
    gla::HdaLin &m = p.lin[0];
    m.x.p = q;
    m.y.p = k;
    m.z.p = v;
    m.init = h0;
    m.fin = hT;
    m.out = o;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    size_t states;
    const size_t need = empty ? 0 : hda_workspace(sh, p, opt, path, sms, &states);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dev != GLA_OK && !(opt && opt->workspace)) return (gla_status)dev;
    void *ws = nullptr;
    rc = get_workspace(opt ? opt->workspace : nullptr, opt ? opt->workspace_bytes : 0, need, s, used,
                       7, &ws);
    if (rc != GLA_OK) return rc;
    if (dev != GLA_OK) return (gla_status)dev;
    if (none) return GLA_OK;
    if (empty) return empty_state(hT, h0, d.bs, s);
    return run_hda(p, sh, opt, ws, states, path, sms, err, s);
}

gla_status hda_bwd(const void *d_o, const void *q, const void *k, const void *v,
                   const float *decay, float scale, const float *h0, const float *dhT, void *dq,
                   void *dk, void *dv, float *dh0, const hda_shape *shape, const gla_options *opt,
                   gla_stream_t stream) {
    HdaDims d;
    gla_status rc = hda_dims(shape, false, &d);
    if (rc == GLA_OK) rc = check_options(opt);
    if (rc != GLA_OK) return rc;
    const hda_shape &sh = *shape;
    const bool none = sh.B * sh.H == 0, empty = none || sh.T == 0;
    if (!empty && (!d_o || !q || !k || !v || !decay || !dq || !dk || !dv)) return GLA_ERR_NULL_ARG;
    for (const void *p : {d_o, q, k, v, (const void *)h0, (const void *)dhT, (const void *)dq,
                          (const void *)dk, (const void *)dv, (const void *)dh0})
        if (misaligned(p)) return GLA_ERR_MISALIGNED;
    if (reinterpret_cast<uintptr_t>(decay) & 3u) return GLA_ERR_MISALIGNED;
    const int64_t bt = sh.B * sh.T * d.es;
    const Range used[11] = {{d_o, d.bgo}, {q, d.bq}, {k, d.bk}, {v, d.bv}, {decay, sh.H * 4},
                            {h0, d.bs}, {dhT, d.bs}, {dq, bt * sh.Hq * sh.Dk},
                            {dk, bt * sh.Hk * sh.Dk}, {dv, bt * sh.Hv * sh.Dv}, {dh0, d.bs}};
    if ((rc = check_alias(used + 7, 4, used, 7)) != GLA_OK) return rc;
    gla::HdaProblem p = hda_problem(sh, d, true, scale);
    const int path = hda_path(p, opt);
    if (path < 0) return GLA_ERR_UNSUPPORTED_DIM;
    p.decay = decay;
    const void *xyz[3][3] = {{d_o, v, k}, {v, d_o, q}, {k, q, d_o}};
    void *outs[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
        p.lin[i].x.p = xyz[i][0];
        p.lin[i].y.p = xyz[i][1];
        p.lin[i].z.p = xyz[i][2];
        p.lin[i].init = i == 0 ? h0 : dhT;
        p.lin[i].init_t = i < 2;
        p.lin[i].out = outs[i];
    }
    p.lin[2].fin = dh0;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    size_t states;
    const size_t need = empty ? 0 : hda_workspace(sh, p, opt, path, sms, &states);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dev != GLA_OK && !(opt && opt->workspace)) return (gla_status)dev;
    void *ws = nullptr;
    rc = get_workspace(opt ? opt->workspace : nullptr, opt ? opt->workspace_bytes : 0, need, s, used,
                       11, &ws);
    if (rc != GLA_OK) return rc;
    if (dev != GLA_OK) return (gla_status)dev;
    if (none) return GLA_OK;
    if (empty) return empty_state(dh0, dhT, d.bs, s);
    return run_hda(p, sh, opt, ws, states, path, sms, err, s);
}

gla_status hda_step(const void *q, const void *k, const void *v, const float *decay, float scale,
                    float *S, const int32_t *slots, void *o, int64_t P, const hda_shape *shape,
                    gla_stream_t stream) {
    HdaDims d;
    gla_status rc = hda_dims(shape, true, &d);
    if (rc != GLA_OK) return rc;
    const hda_shape &sh = *shape;
    int64_t pool;
    if (P < 0 || P > (int64_t(1) << 30) || !mul_ok(P, sh.H, &pool) ||
        !mul_ok(pool, sh.Dk * sh.Dv, &pool) || (!slots && P < sh.B))
        return GLA_ERR_BAD_SHAPE;
    const bool empty = sh.B * sh.H == 0;
    if (!empty && (!q || !k || !v || !decay || !o || (!S && pool > 0))) return GLA_ERR_NULL_ARG;
    for (const void *p : {(const void *)S, (const void *)o})
        if (misaligned(p)) return GLA_ERR_MISALIGNED;
    for (const void *p : {q, k, v})
        if (reinterpret_cast<uintptr_t>(p) & (size_t)(d.es - 1)) return GLA_ERR_MISALIGNED;
    if (bad_int(decay) || bad_int(slots)) return GLA_ERR_MISALIGNED;
    const Range used[7] = {{q, d.bq}, {k, d.bk}, {v, d.bv}, {decay, sh.H * 4}, {slots, sh.B * 4},
                           {o, d.bo}, {S, pool * 4}};
    if ((rc = check_alias(used + 5, 2, used, 5)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (empty) return GLA_OK;
    gla::HdaStep p{};
    p.q = d.q;
    p.k = d.k;
    p.v = d.v;
    p.q.p = q;
    p.k.p = k;
    p.v.p = v;
    p.decay = decay;
    p.scale = scale;
    p.S = S;
    p.slots = slots;
    p.o = o;
    p.R = sh.B;
    p.P = P;
    p.H = sh.H;
    p.Dk = (int)sh.Dk;
    p.Dv = (int)sh.Dv;
    p.io = sh.io;
    const cudaError_t e = gla::launch_hda_step(p, sms, err, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("decay step launch", e);
}

size_t gla_group_norm_workspace_size(const gla_norm_shape *shape, int backward) {
    gla::NormProblem p;
    int64_t bx, bg, bdy, by;
    if (norm_problem(shape, &p, &bx, &bg, &bdy, &by) != GLA_OK || by == 0) return 0;
    int sms;
    unsigned *err;
    gla::device_info(&sms, &err);
    return gla::norm_workspace_bytes(p, backward != 0, sms);
}

gla_status gla_group_norm_fwd(const void *x, const float *w, const float *b, const void *gate,
                              void *y, float *mean, float *rstd, const gla_norm_shape *shape,
                              void *workspace, size_t workspace_bytes, gla_stream_t stream) {
    gla::NormProblem p;
    int64_t bx, bg, bdy, by;
    gla_status rc = norm_problem(shape, &p, &bx, &bg, &bdy, &by);
    if (rc != GLA_OK) return rc;
    if (by > 0 && (!x || !y)) return GLA_ERR_NULL_ARG;
    if (misaligned(y) || unaligned(x, p.io) || unaligned(gate, p.io) || bad_int(w) || bad_int(b) ||
        bad_int(mean) || bad_int(rstd))
        return GLA_ERR_MISALIGNED;
    const Range used[7] = {{x, bx}, {w, p.C * 4}, {b, p.C * 4}, {gate, gate ? bg : 0}, {y, by},
                           {mean, p.N * p.G * 4}, {rstd, p.N * p.G * 4}};
    if ((rc = check_alias(used + 4, 3, used, 4)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (by == 0) {   // statistics of nothing: 0 / 0 (all bits set is a NaN)
        for (float *d : {mean, rstd}) {
            if (!d || p.N * p.G == 0) continue;
            const cudaError_t e = cudaMemsetAsync(d, 0xff, (size_t)(p.N * p.G) * 4, s);
            if (e != cudaSuccess) return (gla_status)gla::launch_failed("group norm launch", e);
        }
        return GLA_OK;
    }
    p.x = x;
    p.w = w;
    p.b = b;
    p.gate = gate;
    p.y = y;
    p.mean = mean;
    p.rstd = rstd;
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::norm_workspace_bytes(p, false, sms), s, used,
                       7, &ws);
    if (rc != GLA_OK) return rc;
    const cudaError_t e = gla::launch_norm_fwd(p, ws, sms, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("group norm launch", e);
}

gla_status gla_group_norm_bwd(const void *dy, const void *x, const float *mean, const float *rstd,
                              const float *w, const float *b, const void *gate, void *dx,
                              float *dw, float *db, void *dgate, const gla_norm_shape *shape,
                              void *workspace, size_t workspace_bytes, gla_stream_t stream) {
    gla::NormProblem p;
    int64_t bx, bg, bdy, by;
    gla_status rc = norm_problem(shape, &p, &bx, &bg, &bdy, &by);
    if (rc != GLA_OK) return rc;
    if (by > 0 && (!dy || !x || !mean || !rstd || !dx || (gate && !dgate))) return GLA_ERR_NULL_ARG;
    if (misaligned(dx) || misaligned(dgate) || unaligned(x, p.io) || unaligned(gate, p.io) ||
        unaligned(dy, p.io) || bad_int(w) || bad_int(b) || bad_int(mean) || bad_int(rstd) ||
        bad_int(dw) || bad_int(db))
        return GLA_ERR_MISALIGNED;
    const Range used[11] = {{x, bx}, {w, p.C * 4}, {b, p.C * 4}, {gate, gate ? bg : 0}, {dy, bdy},
                            {mean, p.N * p.G * 4}, {rstd, p.N * p.G * 4}, {dx, by}, {dw, p.C * 4},
                            {db, p.C * 4}, {dgate, gate ? by : 0}};
    if ((rc = check_alias(used + 7, 4, used, 7)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (by == 0) {   // nothing to sum
        for (float *d : {dw, db}) {
            if (!d || p.C == 0) continue;
            const cudaError_t e = cudaMemsetAsync(d, 0, (size_t)p.C * 4, s);
            if (e != cudaSuccess) return (gla_status)gla::launch_failed("group norm launch", e);
        }
        return GLA_OK;
    }
    p.x = x;
    p.dy = dy;
    p.w = w;
    p.b = b;
    p.gate = gate;
    p.mean = const_cast<float *>(mean);
    p.rstd = const_cast<float *>(rstd);
    p.dx = dx;
    p.dw = dw;
    p.db = db;
    p.dgate = dgate;
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::norm_workspace_bytes(p, true, sms), s, used,
                       11, &ws);
    if (rc != GLA_OK) return rc;
    const cudaError_t e = gla::launch_norm_bwd(p, ws, sms, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("group norm launch", e);
}

gla_status gla_pages_copy(void *pool, int64_t P, int64_t page_bytes, const int32_t *src,
                          const int32_t *dst, int64_t n, gla_stream_t stream) {
    gla_status rc = check_pool(pool, P, page_bytes);
    if (rc != GLA_OK) return rc;
    if (n < 0 || n > (int64_t(1) << 30)) return GLA_ERR_BAD_SHAPE;
    if (n > 0 && (!src || !dst)) return GLA_ERR_NULL_ARG;
    if (bad_int(src) || bad_int(dst)) return GLA_ERR_MISALIGNED;
    const Range out{pool, P * page_bytes}, ins[2] = {{src, n * 4}, {dst, n * 4}};
    if ((rc = check_alias(&out, 1, ins, 2)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n == 0 || page_bytes == 0) return GLA_OK;
    gla::PagePool p{pool, P, page_bytes, nullptr, 0, 0, nullptr, nullptr};
    const cudaError_t e = gla::launch_pages_copy(p, src, dst, n, sms, err,
                                                 reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("page copy launch", e);
}

size_t gla_pages_workspace_size(int64_t P, int64_t R, int64_t M, int64_t n) {
    int64_t e;
    if (P < 0 || P > (int64_t(1) << 30) || R < 0 || R > (int64_t(1) << 30) || !mul_ok(n, M, &e) ||
        e > (int64_t(1) << 30) || n > (int64_t(1) << 30))
        return 0;
    const gla::PagePool p{nullptr, P, 0, nullptr, R, M, nullptr, nullptr};
    return std::max({n > 0 ? gla::pages_fork_workspace(p, n) : 0, n > 0 ? gla::pages_free_workspace(p) : 0,
                     P > 0 ? gla::pages_compact_workspace(p) : 0});
}

gla_status gla_pages_fork_ex(void *pool, int64_t P, int64_t page_bytes, int32_t *table, int64_t R,
                             int64_t M, int32_t *free_stack, int32_t *count, const int32_t *parents,
                             const int32_t *children, int64_t n, void *workspace,
                             size_t workspace_bytes, gla_stream_t stream) {
    gla_status rc = check_pool(pool, P, page_bytes);
    if (rc == GLA_OK) rc = check_table(P, table, R, M, free_stack, count, n);
    if (rc != GLA_OK) return rc;
    if (n > 0 && (!parents || !children)) return GLA_ERR_NULL_ARG;
    if (bad_int(parents) || bad_int(children)) return GLA_ERR_MISALIGNED;
    const Range used[6] = {{parents, n * 4}, {children, n * 4}, {pool, P * page_bytes}, {table, R * M * 4},
                           {free_stack, P * 4}, {count, 4}};
    if ((rc = check_alias(used + 2, 4, used, 2)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n * M == 0) return GLA_OK;
    gla::PagePool p{pool, P, page_bytes, table, R, M, free_stack, count};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::pages_fork_workspace(p, n), s, used, 6, &ws);
    if (rc != GLA_OK) return rc;
    const cudaError_t e = gla::launch_pages_fork(p, parents, children, n, ws, sms, err, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("page fork launch", e);
}

gla_status gla_pages_fork(void *pool, int64_t P, int64_t page_bytes, int32_t *table, int64_t R,
                          int64_t M, int32_t *free_stack, int32_t *count, const int32_t *parents,
                          const int32_t *children, int64_t n, gla_stream_t stream) {
    return gla_pages_fork_ex(pool, P, page_bytes, table, R, M, free_stack, count, parents, children, n,
                             nullptr, 0, stream);
}

gla_status gla_pages_free_ex(int64_t P, int32_t *table, int64_t R, int64_t M, int32_t *free_stack,
                             int32_t *count, const int32_t *rows, int64_t n, void *workspace,
                             size_t workspace_bytes, gla_stream_t stream) {
    gla_status rc = check_table(P, table, R, M, free_stack, count, n);
    if (rc != GLA_OK) return rc;
    if (n > 0 && !rows) return GLA_ERR_NULL_ARG;
    if (bad_int(rows)) return GLA_ERR_MISALIGNED;
    const Range used[4] = {{rows, n * 4}, {table, R * M * 4}, {free_stack, P * 4}, {count, 4}};
    if ((rc = check_alias(used + 1, 3, used, 1)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n * M == 0) return GLA_OK;
    gla::PagePool p{nullptr, P, 0, table, R, M, free_stack, count};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::pages_free_workspace(p), s, used, 4, &ws);
    if (rc != GLA_OK) return rc;
    const cudaError_t e = gla::launch_pages_free(p, rows, n, ws, err, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("page free launch", e);
}

gla_status gla_pages_free(int64_t P, int32_t *table, int64_t R, int64_t M, int32_t *free_stack,
                          int32_t *count, const int32_t *rows, int64_t n, gla_stream_t stream) {
    return gla_pages_free_ex(P, table, R, M, free_stack, count, rows, n, nullptr, 0, stream);
}

gla_status gla_pages_compact_ex(void *pool, int64_t P, int64_t page_bytes, int32_t *table, int64_t R,
                                int64_t M, int32_t *free_stack, int32_t *count, void *workspace,
                                size_t workspace_bytes, gla_stream_t stream) {
    gla_status rc = check_pool(pool, P, page_bytes);
    if (rc == GLA_OK) rc = check_table(P, table, R, M, free_stack, count, 0);
    if (rc != GLA_OK) return rc;
    const Range outs[4] = {{pool, P * page_bytes}, {table, R * M * 4}, {free_stack, P * 4}, {count, 4}};
    if ((rc = check_alias(outs, 4, nullptr, 0)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (P == 0) return GLA_OK;
    gla::PagePool p{pool, P, page_bytes, table, R, M, free_stack, count};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::pages_compact_workspace(p), s, outs, 4, &ws);
    if (rc != GLA_OK) return rc;
    const cudaError_t e = gla::launch_pages_compact(p, ws, sms, err, s);
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed("page compaction launch", e);
}

gla_status gla_pages_compact(void *pool, int64_t P, int64_t page_bytes, int32_t *table, int64_t R,
                             int64_t M, int32_t *free_stack, int32_t *count, gla_stream_t stream) {
    return gla_pages_compact_ex(pool, P, page_bytes, table, R, M, free_stack, count, nullptr, 0, stream);
}

}  // extern "C"
