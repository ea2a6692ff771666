// C ABI of the operators around a recurrent layer: the short convolution (gla_conv_*), the selective
// state space scan (ssm_*), the norm and rotation of queries and keys (gla_qk_norm_*). Argument
// checks and workspaces; include/gla.h has the contracts.
#include <algorithm>

#include "api_util.h"
#include "conv.h"
#include "gla.h"
#include "gla_internal.h"
#include "qk_norm.h"
#include "ssm.h"

namespace {

using namespace gla::api;

constexpr int64_t kMostRows = int64_t(1) << 30;     // tokens, rows, heads of a call

// Strides of [B, T, width] rows (contiguous where the caller's are both zero) and their extent in
// bytes. Dimensions of one element take the stride of a packed tensor, whatever the caller's says.
bool rows_of(const gla_rows &in, int64_t B, int64_t T, int64_t width, int es, int64_t *sb, int64_t *st,
             int64_t *bytes) {
    const bool packed = in.b == 0 && in.t == 0;
    *st = packed || T <= 1 ? width : in.t;
    *sb = packed || B <= 1 ? std::max<int64_t>(T, 1) * width : in.b;
    *bytes = 0;
    if (B == 0 || T == 0 || width == 0) return true;
    int64_t a, b;
    if (*st <= 0 || *sb <= 0 || !mul_ok(B - 1, *sb, &a) || !mul_ok(T - 1, *st, &b)) return false;
    if (a + b > kMostElems / 16 - width) return false;
    *bytes = (a + b + width) * es;
    return true;
}

// The same of [B, T, heads, D].
bool heads_of(const gla_strides &in, int64_t B, int64_t T, int64_t heads, int64_t D, int es, int64_t *sb,
              int64_t *st, int64_t *sh, int64_t *bytes) {
    const bool packed = in.b == 0 && in.t == 0 && in.h == 0;
    *sh = packed || heads <= 1 ? D : in.h;
    *st = packed || T <= 1 ? heads * D : in.t;
    *sb = packed || B <= 1 ? std::max<int64_t>(T, 1) * heads * D : in.b;
    *bytes = 0;
    if (B == 0 || T == 0 || heads == 0) return true;
    int64_t a, b, c;
    if (*sh <= 0 || *st <= 0 || *sb <= 0 || !mul_ok(B - 1, *sb, &a) || !mul_ok(T - 1, *st, &b) ||
        !mul_ok(heads - 1, *sh, &c))
        return false;
    if (a > kMostElems / 16 || b > kMostElems / 16 || a + b + c > kMostElems / 16 - D) return false;
    *bytes = (a + b + c + D) * es;
    return true;
}

int elem_size(int io) { return io == GLA_IO_BF16 ? 2 : 4; }
bool bad_io(int io) { return io != GLA_IO_BF16 && io != GLA_IO_F32; }

gla_status done(const char *what, cudaError_t e) {
    return e == cudaSuccess ? GLA_OK : (gla_status)gla::launch_failed(what, e);
}
cudaStream_t cuda_stream(gla_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Clears n bytes at p, if there are any.
gla_status clear(void *p, int64_t n, const char *what, cudaStream_t s) {
    return p && n > 0 ? done(what, cudaMemsetAsync(p, 0, (size_t)n, s)) : GLA_OK;
}

// ---------------------------------------------------------------- convolution
struct ConvSizes {
    int64_t x, dy, y, state;        // bytes
};

gla_status conv_problem(const gla_conv_shape *sh, bool step, gla::ConvProblem *p, ConvSizes *n) {
    if (!sh) return GLA_ERR_NULL_ARG;
    if (bad_io(sh->io) || sh->act < GLA_ACT_NONE || sh->act > GLA_ACT_GELU) return GLA_ERR_BAD_OPTION;
    const int64_t T = step ? 1 : sh->T;
    if (sh->B < 0 || T < 0 || sh->C < 0 || sh->B > kMostRows || T > kMostRows || sh->C > (int64_t(1) << 20))
        return GLA_ERR_BAD_SHAPE;
    if (sh->W < 1 || sh->W > 8) return GLA_ERR_UNSUPPORTED_DIM;
    const int es = elem_size(sh->io);
    int64_t e;
    if (!mul_ok(sh->B, T, &e) || e > (int64_t(1) << 33) || !mul_ok(e, sh->C, &e) || e > (int64_t(1) << 37))
        return GLA_ERR_BAD_SHAPE;
    *p = gla::ConvProblem{};
    n->y = e * es;
    n->state = sh->B * (sh->W - 1) * sh->C * es;
    gla_rows x = sh->x, dy = sh->dy;
    if (step) x.t = x.b ? 1 : 0;        // one token: its stride says nothing
    if (!rows_of(x, sh->B, T, sh->C, es, &p->x_b, &p->x_t, &n->x) ||
        !rows_of(dy, sh->B, T, sh->C, es, &p->dy_b, &p->dy_t, &n->dy))
        return GLA_ERR_BAD_SHAPE;
    p->B = sh->B;
    p->T = T;
    p->C = sh->C;
    p->W = (int)sh->W;
    p->act = sh->act;
    p->io = sh->io;
    return GLA_OK;
}

// ---------------------------------------------------------------- scan
struct SsmSizes {
    int64_t u, dt, z, bm, cm, go, o, rows, state;       // bytes
};

gla_status ssm_problem(const ssm_shape *sh, bool step, gla::SsmProblem *p, SsmSizes *n) {
    if (!sh) return GLA_ERR_NULL_ARG;
    if (bad_io(sh->io) || sh->softplus < 0 || sh->softplus > 1) return GLA_ERR_BAD_OPTION;
    const int64_t T = step ? 1 : sh->T;
    if (sh->B < 0 || T < 0 || sh->C < 0 || sh->B > kMostRows || T > kMostRows || sh->C > (int64_t(1) << 24))
        return GLA_ERR_BAD_SHAPE;
    if (sh->G < 1 || sh->G > (int64_t(1) << 24) || sh->C % sh->G != 0) return GLA_ERR_BAD_SHAPE;
    if (sh->N < 1 || sh->N > 128) return GLA_ERR_UNSUPPORTED_DIM;
    const int es = elem_size(sh->io);
    int64_t e, c;
    // (what the grids of the kernels hold)
    int64_t r;
    if (!mul_ok(sh->B, sh->C, &c) || c > (int64_t(1) << 30) || !mul_ok(c, T, &e) || e > (int64_t(1) << 38) ||
        !mul_ok(sh->B * T, sh->G * (sh->N + 3), &r) || r > (int64_t(1) << 35))
        return GLA_ERR_BAD_SHAPE;
    *p = gla::SsmProblem{};
    n->o = e * es;
    n->rows = sh->B * T * sh->G * sh->N * es;
    n->state = c * sh->N * 4;
    struct One {
        gla_rows in;
        gla::SsmRows *out;
        int64_t width, *bytes;
    };
    const One all[6] = {{sh->u, &p->u, sh->C, &n->u},           {sh->dt, &p->dt, sh->C, &n->dt},
                        {sh->z, &p->z, sh->C, &n->z},           {sh->b, &p->Bm, sh->G * sh->N, &n->bm},
                        {sh->c, &p->Cm, sh->G * sh->N, &n->cm}, {sh->d_o, &p->go, sh->C, &n->go}};
    for (const One &r : all) {
        gla_rows in = r.in;
        if (step) in.t = in.b ? 1 : 0;
        if (!rows_of(in, sh->B, T, r.width, es, &r.out->b, &r.out->t, r.bytes)) return GLA_ERR_BAD_SHAPE;
    }
    p->B = sh->B;
    p->T = T;
    p->C = sh->C;
    p->G = sh->G;
    p->N = (int)sh->N;
    p->softplus = sh->softplus;
    p->io = sh->io;
    return GLA_OK;
}

gla_status ssm_options(const gla_options *opt) {
    if (!opt) return GLA_OK;
    if ((opt->path != GLA_PATH_AUTO && opt->path != GLA_PATH_EXACT) || opt->seq_splits < 0 ||
        opt->gate != GLA_GATE_KEY)
        return GLA_ERR_BAD_OPTION;
    return GLA_OK;
}

size_t ssm_workspace(const ssm_shape *shape, const gla_options *opt, bool backward) {
    gla::SsmProblem p;
    SsmSizes n;
    if (ssm_problem(shape, false, &p, &n) != GLA_OK || ssm_options(opt) != GLA_OK || n.o == 0) return 0;
    int sms;
    unsigned *err;
    gla::device_info(&sms, &err);
    const int splits = opt ? opt->seq_splits : 0;
    return backward ? gla::ssm_bwd_workspace_bytes(p, splits, sms, true) : gla::ssm_fwd_workspace_bytes(p, splits, sms, true);
}

// A state after no tokens: the one before them, or zero.
gla_status no_tokens(float *dst, const float *src, int64_t bytes, cudaStream_t s) {
    if (!dst || bytes == 0) return GLA_OK;
    if (!src) return clear(dst, bytes, "scan of no tokens", s);
    return done("scan of no tokens", cudaMemcpyAsync(dst, src, (size_t)bytes, cudaMemcpyDeviceToDevice, s));
}

// ---------------------------------------------------------------- norm and rotation
struct QkSizes {
    int64_t x[2], go[2], out[2], r[2];      // bytes, of q and k
};

gla_status qk_problem(const gla_qk_shape *sh, gla::QkProblem *p, QkSizes *n) {
    if (!sh) return GLA_ERR_NULL_ARG;
    if (bad_io(sh->io) || sh->norm < GLA_NORM_NONE || sh->norm > GLA_NORM_L2 || sh->pairs < 0 || sh->pairs > 1 ||
        !(sh->eps >= 0.f))
        return GLA_ERR_BAD_OPTION;
    if (sh->B < 0 || sh->T < 0 || sh->Hq < 0 || sh->Hk < 0 || sh->P < 0 || sh->B > kMostRows || sh->T > kMostRows ||
        sh->Hq > 65536 || sh->Hk > 65536 || sh->P > (int64_t(1) << 31) - 1)
        return GLA_ERR_BAD_SHAPE;
    if (sh->D < 1 || sh->D > 1024) return GLA_ERR_UNSUPPORTED_DIM;
    if (sh->R < 0 || sh->R > sh->D || sh->R % 2 != 0) return GLA_ERR_BAD_SHAPE;
    const int es = elem_size(sh->io);
    int64_t bt;
    if (!mul_ok(sh->B, sh->T, &bt) || bt > (int64_t(1) << 33) || bt * (sh->Hq + sh->Hk) > (int64_t(1) << 33))
        return GLA_ERR_BAD_SHAPE;
    *p = gla::QkProblem{};
    const int64_t heads[2] = {sh->Hq, sh->Hk};
    const gla_strides *in[2] = {&sh->q, &sh->k}, *go[2] = {&sh->d_qo, &sh->d_ko};
    for (int i = 0; i < 2; ++i) {
        gla::QkHeads &t = p->t[i];
        t.heads = (int)heads[i];
        n->out[i] = bt * heads[i] * sh->D * es;
        n->r[i] = bt * heads[i] * 4;
        if (!heads_of(*in[i], sh->B, sh->T, heads[i], sh->D, es, &t.x_b, &t.x_t, &t.x_h, &n->x[i]) ||
            !heads_of(*go[i], sh->B, sh->T, heads[i], sh->D, es, &t.g_b, &t.g_t, &t.g_h, &n->go[i]))
            return GLA_ERR_BAD_SHAPE;
    }
    p->B = sh->B;
    p->T = sh->T;
    p->P = sh->P;
    p->D = (int)sh->D;
    p->R = (int)sh->R;
    p->norm = sh->norm;
    p->pairs = sh->pairs;
    p->io = sh->io;
    p->eps = sh->eps;
    return GLA_OK;
}

}  // namespace

extern "C" {

gla_status gla_conv_fwd(const void *x, const float *w, const float *bias, const void *s0, void *y, void *sT,
                        const gla_conv_shape *shape, gla_stream_t stream) {
    gla::ConvProblem p;
    ConvSizes n;
    gla_status rc = conv_problem(shape, false, &p, &n);
    if (rc != GLA_OK) return rc;
    if (n.y > 0 && (!x || !w || !y)) return GLA_ERR_NULL_ARG;
    if (unaligned(x, p.io) || misaligned(s0) || misaligned(y) || misaligned(sT) || bad_int(w) || bad_int(bias))
        return GLA_ERR_MISALIGNED;
    const Range used[6] = {{x, n.x}, {w, p.C * p.W * 4}, {bias, p.C * 4}, {s0, n.state}, {y, n.y}, {sT, n.state}};
    if ((rc = check_alias(used + 4, 2, used, 4)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = cuda_stream(stream);
    if (n.y == 0) {     // no tokens: the last inputs are the first ones
        if (!sT || n.state == 0) return GLA_OK;
        if (!s0) return clear(sT, n.state, "convolution of no tokens", s);
        return done("convolution of no tokens", cudaMemcpyAsync(sT, s0, (size_t)n.state, cudaMemcpyDeviceToDevice, s));
    }
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.s0 = s0;
    p.y = y;
    p.sT = p.W > 1 ? sT : nullptr;
    return done("convolution launch", gla::launch_conv_fwd(p, sms, s));
}

size_t gla_conv_bwd_workspace_size(const gla_conv_shape *shape) {
    gla::ConvProblem p;
    ConvSizes n;
    if (conv_problem(shape, false, &p, &n) != GLA_OK || n.y == 0) return 0;
    int sms;
    unsigned *err;
    gla::device_info(&sms, &err);
    return gla::conv_bwd_workspace_bytes(p, sms);
}

gla_status gla_conv_bwd(const void *dy, const void *x, const float *w, const float *bias, const void *s0,
                        const void *dsT, void *dx, float *dw, float *dbias, void *ds0, const gla_conv_shape *shape,
                        void *workspace, size_t workspace_bytes, gla_stream_t stream) {
    gla::ConvProblem p;
    ConvSizes n;
    gla_status rc = conv_problem(shape, false, &p, &n);
    if (rc != GLA_OK) return rc;
    if (n.y > 0 && (!dy || !x || !w || !dx)) return GLA_ERR_NULL_ARG;
    if (unaligned(x, p.io) || unaligned(dy, p.io) || misaligned(s0) || misaligned(dsT) || misaligned(dx) ||
        misaligned(ds0) || bad_int(w) || bad_int(bias) || bad_int(dw) || bad_int(dbias))
        return GLA_ERR_MISALIGNED;
    const Range used[10] = {{dy, n.dy}, {x, n.x}, {w, p.C * p.W * 4}, {bias, p.C * 4}, {s0, n.state},
                            {dsT, n.state}, {dx, n.y}, {dw, p.C * p.W * 4}, {dbias, p.C * 4}, {ds0, n.state}};
    if ((rc = check_alias(used + 6, 4, used, 6)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = cuda_stream(stream);
    if (n.y == 0) {
        if ((rc = clear(dw, p.C * p.W * 4, "convolution of no tokens", s)) != GLA_OK) return rc;
        if ((rc = clear(dbias, p.C * 4, "convolution of no tokens", s)) != GLA_OK) return rc;
        if (!ds0 || n.state == 0) return GLA_OK;
        if (!dsT) return clear(ds0, n.state, "convolution of no tokens", s);
        return done("convolution of no tokens",
                    cudaMemcpyAsync(ds0, dsT, (size_t)n.state, cudaMemcpyDeviceToDevice, s));
    }
    p.dy = dy;
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.s0 = s0;
    p.dsT = p.W > 1 ? dsT : nullptr;
    p.dx = dx;
    p.dw = dw;
    p.dbias = dbias;
    p.ds0 = p.W > 1 ? ds0 : nullptr;
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::conv_bwd_workspace_bytes(p, sms), s, used, 10, &ws);
    if (rc != GLA_OK) return rc;
    return done("convolution gradient launch", gla::launch_conv_bwd(p, ws, sms, s));
}

gla_status gla_conv_step(const void *x, const float *w, const float *bias, void *S, const int32_t *slots, void *y,
                         int64_t P, const gla_conv_shape *shape, gla_stream_t stream) {
    gla::ConvProblem p;
    ConvSizes n;
    gla_status rc = conv_problem(shape, true, &p, &n);
    if (rc != GLA_OK) return rc;
    int64_t pool;
    if (P < 0 || P > kMostRows || !mul_ok(P, (p.W - 1) * p.C, &pool) || (!slots && P < p.B)) return GLA_ERR_BAD_SHAPE;
    pool *= elem_size(p.io);
    if (n.y > 0 && (!x || !w || !y || (pool > 0 && !S))) return GLA_ERR_NULL_ARG;
    if (unaligned(x, p.io) || misaligned(S) || misaligned(y) || bad_int(w) || bad_int(bias) || bad_int(slots))
        return GLA_ERR_MISALIGNED;
    const Range used[6] = {{x, n.x}, {w, p.C * p.W * 4}, {bias, p.C * 4}, {slots, p.B * 4}, {y, n.y}, {S, pool}};
    if ((rc = check_alias(used + 4, 2, used, 4)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n.y == 0) return GLA_OK;
    p.x = x;
    p.w = w;
    p.bias = bias;
    p.S = S;
    p.slots = slots;
    p.y = y;
    p.P = P;
    return done("convolution step launch", gla::launch_conv_step(p, err, cuda_stream(stream)));
}

size_t ssm_fwd_workspace_size(const ssm_shape *shape, const gla_options *opt) {
    return ssm_workspace(shape, opt, false);
}
size_t ssm_bwd_workspace_size(const ssm_shape *shape, const gla_options *opt) {
    return ssm_workspace(shape, opt, true);
}

gla_status ssm_fwd(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                   const void *z, const float *dt_bias, const float *h0, void *o, float *hT, const ssm_shape *shape,
                   const gla_options *opt, gla_stream_t stream) {
    gla::SsmProblem p;
    SsmSizes n;
    gla_status rc = ssm_problem(shape, false, &p, &n);
    if (rc == GLA_OK) rc = ssm_options(opt);
    if (rc != GLA_OK) return rc;
    if (n.o > 0 && (!u || !dt || !A || !Bm || !Cm || !o)) return GLA_ERR_NULL_ARG;
    for (const void *q : {u, dt, Bm, Cm, z})
        if (unaligned(q, p.io)) return GLA_ERR_MISALIGNED;
    if (misaligned(h0) || misaligned(o) || misaligned(hT) || bad_int(A) || bad_int(D) || bad_int(dt_bias))
        return GLA_ERR_MISALIGNED;
    const Range used[11] = {{u, n.u}, {dt, n.dt}, {A, p.C * p.N * 4}, {Bm, n.bm}, {Cm, n.cm}, {D, p.C * 4},
                            {z, z ? n.z : 0}, {dt_bias, p.C * 4}, {h0, n.state}, {o, n.o}, {hT, n.state}};
    if ((rc = check_alias(used + 9, 2, used, 9)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    cudaStream_t s = cuda_stream(stream);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n.o == 0) return no_tokens(hT, h0, n.state, s);
    p.u.p = u;
    p.dt.p = dt;
    p.A = A;
    p.Bm.p = Bm;
    p.Cm.p = Cm;
    p.D = D;
    p.z.p = z;
    p.dt_bias = dt_bias;
    p.h0 = h0;
    p.o = o;
    p.hT = hT;
    const int splits = opt ? opt->seq_splits : 0;
    void *ws;
    rc = get_workspace(opt ? opt->workspace : nullptr, opt ? opt->workspace_bytes : 0,
                       gla::ssm_fwd_workspace_bytes(p, splits, sms, false), s, used, 11, &ws);
    if (rc != GLA_OK) return rc;
    return done("scan launch", gla::launch_ssm_fwd(p, splits, sms, ws, err, s));
}

gla_status ssm_bwd(const void *d_o, const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                   const float *D, const void *z, const float *dt_bias, const float *h0, const float *dhT, void *du,
                   void *ddt, float *dA, void *dBm, void *dCm, float *dD, void *dz, float *ddt_bias, float *dh0,
                   const ssm_shape *shape, const gla_options *opt, gla_stream_t stream) {
    gla::SsmProblem p;
    SsmSizes n;
    gla_status rc = ssm_problem(shape, false, &p, &n);
    if (rc == GLA_OK) rc = ssm_options(opt);
    if (rc != GLA_OK) return rc;
    if (dz && !z) return GLA_ERR_NULL_ARG;
    if (n.o > 0 && (!d_o || !u || !dt || !A || !Bm || !Cm || !du || !ddt || !dA || !dBm || !dCm))
        return GLA_ERR_NULL_ARG;
    for (const void *q : {d_o, u, dt, Bm, Cm, z})
        if (unaligned(q, p.io)) return GLA_ERR_MISALIGNED;
    for (const void *q : {(const void *)h0, (const void *)dhT, (const void *)du, (const void *)ddt,
                          (const void *)dBm, (const void *)dCm, (const void *)dz, (const void *)dh0})
        if (misaligned(q)) return GLA_ERR_MISALIGNED;
    for (const float *q : {A, D, dt_bias, (const float *)dA, (const float *)dD, (const float *)ddt_bias})
        if (bad_int(q)) return GLA_ERR_MISALIGNED;
    const Range used[20] = {{d_o, n.go}, {u, n.u}, {dt, n.dt}, {A, p.C * p.N * 4}, {Bm, n.bm}, {Cm, n.cm},
                            {D, p.C * 4}, {z, z ? n.z : 0}, {dt_bias, p.C * 4}, {h0, n.state}, {dhT, n.state},
                            {du, n.o}, {ddt, n.o}, {dA, p.C * p.N * 4}, {dBm, n.rows}, {dCm, n.rows}, {dD, p.C * 4},
                            {dz, n.o}, {ddt_bias, p.C * 4}, {dh0, n.state}};
    if ((rc = check_alias(used + 11, 9, used, 11)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = cuda_stream(stream);
    if (n.o == 0) {
        const char *what = "scan of no tokens";
        if ((rc = clear(dA, p.C * p.N * 4, what, s)) != GLA_OK) return rc;
        if ((rc = clear(dD, p.C * 4, what, s)) != GLA_OK) return rc;
        if ((rc = clear(ddt_bias, p.C * 4, what, s)) != GLA_OK) return rc;
        if (p.C == 0) {     // tokens without channels
            if ((rc = clear(dBm, n.rows, what, s)) != GLA_OK) return rc;
            if ((rc = clear(dCm, n.rows, what, s)) != GLA_OK) return rc;
        }
        return no_tokens(dh0, dhT, n.state, s);
    }
    p.go.p = d_o;
    p.u.p = u;
    p.dt.p = dt;
    p.A = A;
    p.Bm.p = Bm;
    p.Cm.p = Cm;
    p.D = D;
    p.z.p = z;
    p.dt_bias = dt_bias;
    p.h0 = h0;
    p.dhT = dhT;
    p.du = du;
    p.ddt = ddt;
    p.dA = dA;
    p.dBm = dBm;
    p.dCm = dCm;
    p.dD = dD;
    p.dz = dz;
    p.dbias = ddt_bias;
    p.dh0 = dh0;
    const int splits = opt ? opt->seq_splits : 0;
    void *ws;
    rc = get_workspace(opt ? opt->workspace : nullptr, opt ? opt->workspace_bytes : 0,
                       gla::ssm_bwd_workspace_bytes(p, splits, sms, false), s, used, 20, &ws);
    if (rc != GLA_OK) return rc;
    return done("scan gradient launch", gla::launch_ssm_bwd(p, splits, sms, ws, err, s));
}

gla_status ssm_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                    const void *z, const float *dt_bias, float *S, const int32_t *slots, void *o, int64_t P,
                    const ssm_shape *shape, gla_stream_t stream) {
    gla::SsmProblem p;
    SsmSizes n;
    gla_status rc = ssm_problem(shape, true, &p, &n);
    if (rc != GLA_OK) return rc;
    int64_t pool;
    if (P < 0 || P > kMostRows || !mul_ok(P, p.C * p.N, &pool) || (!slots && P < p.B)) return GLA_ERR_BAD_SHAPE;
    if (n.o > 0 && (!u || !dt || !A || !Bm || !Cm || !o || (pool > 0 && !S))) return GLA_ERR_NULL_ARG;
    for (const void *q : {u, dt, Bm, Cm, z})
        if (unaligned(q, p.io)) return GLA_ERR_MISALIGNED;
    if (misaligned(S) || misaligned(o) || bad_int(A) || bad_int(D) || bad_int(dt_bias) || bad_int(slots))
        return GLA_ERR_MISALIGNED;
    const Range used[11] = {{u, n.u}, {dt, n.dt}, {A, p.C * p.N * 4}, {Bm, n.bm}, {Cm, n.cm}, {D, p.C * 4},
                            {z, z ? n.z : 0}, {dt_bias, p.C * 4}, {slots, p.B * 4}, {o, n.o}, {S, pool * 4}};
    if ((rc = check_alias(used + 9, 2, used, 9)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n.o == 0) return GLA_OK;
    p.u.p = u;
    p.dt.p = dt;
    p.A = A;
    p.Bm.p = Bm;
    p.Cm.p = Cm;
    p.D = D;
    p.z.p = z;
    p.dt_bias = dt_bias;
    p.S = S;
    p.slots = slots;
    p.o = o;
    p.P = P;
    return done("scan step launch", gla::launch_ssm_step(p, sms, err, cuda_stream(stream)));
}

gla_status gla_qk_norm_fwd(const void *q, const void *k, const float *wq, const float *wk, const float *cos,
                           const float *sin, const int32_t *positions, void *qo, void *ko, float *rq, float *rk,
                           const gla_qk_shape *shape, gla_stream_t stream) {
    gla::QkProblem p;
    QkSizes n;
    gla_status rc = qk_problem(shape, &p, &n);
    if (rc != GLA_OK) return rc;
    if (p.norm == GLA_NORM_NONE && (wq || wk)) return GLA_ERR_BAD_OPTION;
    if ((n.out[0] > 0 && (!q || !qo)) || (n.out[1] > 0 && (!k || !ko))) return GLA_ERR_NULL_ARG;
    if (n.out[0] + n.out[1] > 0 && p.R > 0 && p.P > 0 && (!cos || !sin)) return GLA_ERR_NULL_ARG;
    if (unaligned(q, p.io) || unaligned(k, p.io) || misaligned(qo) || misaligned(ko)) return GLA_ERR_MISALIGNED;
    for (const void *f : {(const void *)wq, (const void *)wk, (const void *)cos, (const void *)sin,
                          (const void *)positions, (const void *)rq, (const void *)rk})
        if (bad_int(f)) return GLA_ERR_MISALIGNED;
    const int64_t table = p.P * (p.R / 2) * 4;
    const Range used[11] = {{q, n.x[0]}, {k, n.x[1]}, {wq, p.D * 4}, {wk, p.D * 4}, {cos, table}, {sin, table},
                            {positions, p.B * p.T * 4}, {qo, n.out[0]}, {ko, n.out[1]}, {rq, n.r[0]}, {rk, n.r[1]}};
    if ((rc = check_alias(used + 7, 4, used, 7)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    if (n.out[0] + n.out[1] == 0) return GLA_OK;
    p.t[0].x = q;
    p.t[1].x = k;
    p.t[0].w = wq;
    p.t[1].w = wk;
    p.t[0].out = qo;
    p.t[1].out = ko;
    p.t[0].r = p.norm ? rq : nullptr;
    p.t[1].r = p.norm ? rk : nullptr;
    p.cos = cos;
    p.sin = sin;
    p.positions = positions;
    return done("norm and rotation launch", gla::launch_qk_fwd(p, sms, err, cuda_stream(stream)));
}

size_t gla_qk_norm_bwd_workspace_size(const gla_qk_shape *shape) {
    gla::QkProblem p;
    QkSizes n;
    if (qk_problem(shape, &p, &n) != GLA_OK || n.out[0] + n.out[1] == 0) return 0;
    int sms;
    unsigned *err;
    gla::device_info(&sms, &err);
    return gla::qk_bwd_workspace_bytes(p, sms);
}

gla_status gla_qk_norm_bwd(const void *d_qo, const void *d_ko, const void *q, const void *k, const float *rq,
                           const float *rk, const float *wq, const float *wk, const float *cos, const float *sin,
                           const int32_t *positions, void *dq, void *dk, float *dwq, float *dwk,
                           const gla_qk_shape *shape, void *workspace, size_t workspace_bytes, gla_stream_t stream) {
    gla::QkProblem p;
    QkSizes n;
    gla_status rc = qk_problem(shape, &p, &n);
    if (rc != GLA_OK) return rc;
    if (p.norm == GLA_NORM_NONE && (wq || wk || dwq || dwk)) return GLA_ERR_BAD_OPTION;
    if ((n.out[0] > 0 && (!d_qo || !q || !dq || (p.norm && !rq))) ||
        (n.out[1] > 0 && (!d_ko || !k || !dk || (p.norm && !rk))))
        return GLA_ERR_NULL_ARG;
    if (n.out[0] + n.out[1] > 0 && p.R > 0 && p.P > 0 && (!cos || !sin)) return GLA_ERR_NULL_ARG;
    for (const void *x : {d_qo, d_ko, q, k})
        if (unaligned(x, p.io)) return GLA_ERR_MISALIGNED;
    if (misaligned(dq) || misaligned(dk)) return GLA_ERR_MISALIGNED;
    for (const void *f : {(const void *)wq, (const void *)wk, (const void *)cos, (const void *)sin,
                          (const void *)positions, (const void *)rq, (const void *)rk, (const void *)dwq,
                          (const void *)dwk})
        if (bad_int(f)) return GLA_ERR_MISALIGNED;
    const int64_t table = p.P * (p.R / 2) * 4;
    const Range used[15] = {{d_qo, n.go[0]}, {d_ko, n.go[1]}, {q, n.x[0]}, {k, n.x[1]}, {rq, n.r[0]}, {rk, n.r[1]},
                            {wq, p.D * 4}, {wk, p.D * 4}, {cos, table}, {sin, table}, {positions, p.B * p.T * 4},
                            {dq, n.out[0]}, {dk, n.out[1]}, {dwq, p.D * 4}, {dwk, p.D * 4}};
    if ((rc = check_alias(used + 11, 4, used, 11)) != GLA_OK) return rc;
    int sms;
    unsigned *err;
    const int dev = gla::device_info(&sms, &err);
    if (dev != GLA_OK) return (gla_status)dev;
    cudaStream_t s = cuda_stream(stream);
    if (n.out[0] + n.out[1] == 0) {
        rc = clear(dwq, p.D * 4, "norm of no heads", s);
        return rc == GLA_OK ? clear(dwk, p.D * 4, "norm of no heads", s) : rc;
    }
    const void *xs[2] = {q, k}, *gos[2] = {d_qo, d_ko};
    const float *rs[2] = {rq, rk}, *ws_[2] = {wq, wk};
    void *outs[2] = {dq, dk};
    float *dws[2] = {dwq, dwk};
    for (int i = 0; i < 2; ++i) {
        p.t[i].x = xs[i];
        p.t[i].go = gos[i];
        p.t[i].r = const_cast<float *>(rs[i]);
        p.t[i].w = ws_[i];
        p.t[i].out = outs[i];
        p.t[i].dw = dws[i];
    }
    p.cos = cos;
    p.sin = sin;
    p.positions = positions;
    void *ws;
    rc = get_workspace(workspace, workspace_bytes, gla::qk_bwd_workspace_bytes(p, sms), s, used, 15, &ws);
    if (rc != GLA_OK) return rc;
    return done("norm and rotation gradient launch", gla::launch_qk_bwd(p, ws, sms, err, s));
}

}  // extern "C"
