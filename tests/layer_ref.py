"""64-bit forms of the short convolution, the selective scan and the norm of queries and keys, with
bounds on what fp32 arithmetic may be off by (CPU, token by token).

U = 2^-24 is the rounding of an fp32 operation. Bounds follow the formulas: |x y| and sums carry the
errors of their parts plus one U of the absolute result for each operation. bf16 results may be
2^-8 of the value (half a step) further off. The hardware's approximate exponential and reciprocal,
which bf16 calls use for the logistic function, are good to 2^-20; e^x by the hardware's 2^x to
2^-21.5 plus the rounding of its argument.
"""
import torch

U = 2.0 ** -24
EXP = 2.0 ** -21.5


def draw(gen, *shape, io="f32", std=1.0):
    t = torch.randn(*shape, generator=gen) * std
    return t.to(torch.bfloat16) if io == "bf16" else t


def gpu(t):
    """The tensor with its strides on the GPU, other memory around it left out."""
    if t is None:
        return None
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return out.copy_(t)


def close(name, got, want, bound):
    """|got - want| <= bound (+ half a step of got's type where that is bf16)."""
    got = got.detach().cpu()
    assert got.shape == want.shape, f"{name}: shape {tuple(got.shape)}, expected {tuple(want.shape)}"
    if got.numel() == 0:
        return
    assert torch.isfinite(want).all(), f"{name}: the 64-bit form is not finite"
    bound = bound + 1e-37
    if got.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    err = (got.double() - want).abs()
    worst = (err / bound).max().item()
    assert worst <= 1, f"{name}: {worst:.3g} times its bound (error {err.max().item():.3g})"


def act64(x, act):
    """act(x) and its derivative."""
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * (1 - s))
    if act == "gelu":
        phi = 0.5 * (1 + torch.erf(x * 0.5 ** 0.5))
        return x * phi, phi + x * torch.exp(-0.5 * x * x) / (2 * torch.pi) ** 0.5
    return x, torch.ones_like(x)


def act_err(io):
    """Relative error of a logistic factor."""
    return 2.0 ** -20 if io == "bf16" else 16 * U


# ---------------------------------------------------------------- convolution
def conv(x, w, bias, s0, dy, dsT, act, io):
    """{name: (value, bound)} of y, sT, dx, dw, db, ds0."""
    x, w = x.double(), w.double()
    B, T, C = x.shape
    W = w.shape[1]
    b = torch.zeros(C).double() if bias is None else bias.double()
    s0 = torch.zeros(B, W - 1, C).double() if s0 is None else s0.double()
    xs = torch.cat((s0, x), 1)
    a = b + sum(w[:, j] * xs[:, j:j + T] for j in range(W))
    size = b.abs() + sum((w[:, j] * xs[:, j:j + T]).abs() for j in range(W))
    ea = (W + 2) * U * size
    y, slope = act64(a, act)
    # slopes of the activations stay below 1.13, those of the slopes below 0.8
    out = dict(y=(y, 1.13 * ea + (act_err(io) + 4 * U) * (y.abs() + U)), sT=(xs[:, T:], 0 * xs[:, T:]))
    if dy is None:
        return out
    dy = dy.double()
    da = dy * slope
    eda = dy.abs() * (0.8 * ea + 4 * act_err(io) * (1 + a.abs()) + 4 * U)
    if act == "none":
        eda = 0 * eda
    dxs, edx = torch.zeros_like(xs), torch.zeros_like(xs)
    if dsT is not None:
        dxs[:, T:] += dsT.double()
    size = dxs.abs()
    for j in range(W):
        dxs[:, j:j + T] += w[:, j] * da
        size[:, j:j + T] += (w[:, j] * da).abs()
        edx[:, j:j + T] += w[:, j].abs() * eda
    edx += (W + 3) * U * size
    n = B * T + 16                  # roundings of a sum over all tokens, in any order
    dw = torch.stack([(da * xs[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    edw = torch.stack([((eda + n * U * da.abs()) * xs[:, j:j + T].abs()).sum((0, 1)) for j in range(W)], 1)
    out.update(dx=(dxs[:, W - 1:], edx[:, W - 1:]), ds0=(dxs[:, :W - 1], edx[:, :W - 1]), dw=(dw, edw),
               db=(da.sum((0, 1)), (eda + n * U * da.abs()).sum((0, 1))))
    return out


# ---------------------------------------------------------------- scan
def scan(d, softplus=True, io="f32", back=True):
    """{name: (value, bound)} of o, hT and the gradients; d: dict of u, dt, A, Bm, Cm, D, z, dt_bias, h0,
    do, dhT (None where not given)."""
    f = {n: None if d.get(n) is None else d[n].double() for n in
         ("u", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "h0", "do", "dhT")}
    u, A = f["u"], f["A"]
    B, T, C = u.shape
    G, N = f["Bm"].shape[2:]
    at = torch.arange(C) // (C // G)
    Bw, Cw = f["Bm"][:, :, at], f["Cm"][:, :, at]                     # [B, T, C, N]
    bias = torch.zeros(C).double() if f["dt_bias"] is None else f["dt_bias"]
    D = torch.zeros(C).double() if f["D"] is None else f["D"]
    raw = f["dt"] + bias
    delta = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    # softplus changes by at most its argument's error times its slope (below min(1, e^x) and
    # delta), and is itself good to 12 U
    ed = (12 * U * delta + U * raw.abs() * delta.clamp(max=1)) if softplus else U * raw.abs()
    p = delta[..., None] * A
    a = torch.exp(p)
    ea = a * (EXP + 3 * U * p.abs()) + a * A.abs() * ed[..., None]    # A log2 e, the product, the step
    b = (delta * u)[..., None] * Bw
    eb = 3 * U * b.abs() + (ed * u.abs())[..., None] * Bw.abs()
    h0 = torch.zeros(B, C, N).double() if f["h0"] is None else f["h0"]
    hs, es = [h0], [torch.zeros_like(h0)]
    for t in range(T):
        h = a[:, t] * hs[-1] + b[:, t]
        size = a[:, t] * hs[-1].abs() + b[:, t].abs()
        es.append((a[:, t] + ea[:, t]) * es[-1] + ea[:, t] * hs[-1].abs() + eb[:, t] + 2 * U * size)
        hs.append(h)
    h, eh = torch.stack(hs, 1), torch.stack(es, 1)                     # [B, T + 1, C, N]
    n = (N + 6) * U
    y = (Cw * h[:, 1:]).sum(3) + D * u
    ey = (Cw.abs() * (eh[:, 1:] + n * h[:, 1:].abs())).sum(3) + 3 * U * (D * u).abs()
    s = act_err(io)
    if f["z"] is None:
        gate, egate = torch.ones_like(u), torch.zeros_like(u)
    else:
        gate = f["z"] * torch.sigmoid(f["z"])
        egate = (s + 4 * U) * gate.abs()
    out = dict(o=(y * gate, ey * gate.abs() + y.abs() * egate + 2 * U * (y * gate).abs()), hT=(h[:, T], eh[:, T]))
    if not back:
        return out
    do = f["do"]
    dy = do * gate
    edy = do.abs() * egate + 2 * U * dy.abs()
    if f["z"] is not None:
        slope = act64(f["z"], "silu")[1]
        ez = 4 * s * (1 + f["z"].abs()) + 8 * U
        out["dz"] = (do * y * slope, do.abs() * (ey * slope.abs() + y.abs() * ez) + 3 * U * (do * y * slope).abs())
    g = torch.zeros(B, C, N).double() if f["dhT"] is None else f["dhT"]
    eg = torch.zeros_like(g)
    names = ("du", "ddt", "dB", "dC")
    val = {k: [None] * T for k in names}
    err = {k: [None] * T for k in names}
    dA, edA = torch.zeros_like(A), torch.zeros_like(A)
    share = lambda x: x.unflatten(1, (G, C // G)).sum(2)       # noqa: E731
    rows, cols = (B * T + 16) * U, (C + 16) * U                 # roundings of the long sums, in any order
    for t in range(T - 1, -1, -1):
        c, bt = Cw[:, t], Bw[:, t]
        x, ut, dt, e_dt = dy[:, t, :, None], u[:, t, :, None], delta[:, t, :, None], ed[:, t, :, None]
        eg = eg + c.abs() * edy[:, t, :, None] + 2 * U * (g.abs() + (c * x).abs())
        g = g + c * x
        gp = a[:, t] * g
        egp = ea[:, t] * g.abs() + (a[:, t] + ea[:, t]) * eg + U * gp.abs()
        w = gp * h[:, t]
        ew = egp * h[:, t].abs() + gp.abs() * eh[:, t] + egp * eh[:, t] + U * w.abs()
        gb = (g * bt).sum(2, keepdim=True)
        egb = (eg * bt.abs() + n * (g * bt).abs()).sum(2, keepdim=True)
        wa = (w * A).sum(2, keepdim=True)
        ewa = (ew * A.abs() + (n + 3 * U) * (w * A).abs()).sum(2, keepdim=True)
        dd = wa + ut * gb
        edd = ewa + ut.abs() * egb + 3 * U * (wa.abs() + (ut * gb).abs())
        sg = torch.sigmoid(raw[:, t, :, None]) if softplus else torch.ones_like(dd)
        val["ddt"][t] = (dd * sg).squeeze(2)
        err["ddt"][t] = (edd * sg + dd.abs() * sg * (16 * U + U * raw[:, t, :, None].abs())).squeeze(2)
        val["du"][t] = (dt * gb).squeeze(2) + D * dy[:, t]
        err["du"][t] = ((e_dt + 3 * U * dt) * gb.abs() + dt * egb + e_dt * egb).squeeze(2).abs() \
            + D.abs() * edy[:, t] + 3 * U * (D * dy[:, t]).abs()
        dA += (w * dt).sum(0)
        edA += (ew * dt.abs() + w.abs() * e_dt + rows * (w * dt).abs()).sum(0)
        v = g * (dt * ut)
        val["dB"][t] = share(v)
        err["dB"][t] = share(eg * (dt * ut).abs() + g.abs() * e_dt * ut.abs() + (cols + 3 * U) * v.abs())
        v = h[:, t + 1] * x
        val["dC"][t] = share(v)
        err["dC"][t] = share(eh[:, t + 1] * x.abs() + h[:, t + 1].abs() * edy[:, t, :, None] + (cols + 3 * U) * v.abs())
        g, eg = gp, egp
    for k in names:
        shape = {"du": (B, 0, C), "ddt": (B, 0, C)}.get(k, (B, 0, G, N))
        if T:
            out[k] = (torch.stack(val[k], 1), torch.stack(err[k], 1))
        else:
            out[k] = (torch.zeros(shape).double(), torch.zeros(shape).double())
    out["dA"] = (dA, edA)
    out["dD"] = ((dy * u).sum((0, 1)), ((edy + rows * dy.abs()) * u.abs()).sum((0, 1)))
    out["dbias"] = (out["ddt"][0].sum((0, 1)), (out["ddt"][1] + rows * out["ddt"][0].abs()).sum((0, 1)))
    out["dh0"] = (g, eg)
    return out


# ---------------------------------------------------------------- norm and rotation
def turn(v, cos, sin, pairs, back=False):
    """The rotation of v [..., D] by cos, sin [..., R / 2] and the sum of its absolute terms."""
    R = 2 * cos.shape[-1]
    if back:
        sin = -sin
    i = torch.arange(R)
    ia, ib = (i[0::2], i[1::2]) if pairs else (i[:R // 2], i[R // 2:])
    out, size = v.clone(), v.abs()
    a, b = v[..., ia], v[..., ib]
    out[..., ia], out[..., ib] = a * cos - b * sin, b * cos + a * sin
    size[..., ia], size[..., ib] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return out, size


def qk(x, w, cos, sin, positions, norm, pairs, eps, go=None, r32=None):
    """{name: (value, bound)} of out, r, and with go (the gradient of out, r32: the forward's factor) dx and dw.
    cos, sin [P, R / 2] or None; positions [B, T]."""
    x = x.double()
    B, T, H, D = x.shape
    s = 1.0 / D if norm == "rms" else 1.0
    ww = torch.ones(D).double() if w is None else w.double()
    r = torch.ones(B, T, H).double() if norm == "none" else (s * (x * x).sum(-1) + eps) ** -0.5
    er = 0 * r if norm == "none" else (D + 16) * U * r             # a sum of D squares, its root
    if cos is not None:
        bad = (positions < 0) | (positions >= cos.shape[0])
        at = positions.long().clamp(0, max(cos.shape[0] - 1, 0))
        c, sn = cos.double()[at][:, :, None], sin.double()[at][:, :, None]
        keep = (~bad).double()[:, :, None]
    else:
        c = sn = torch.zeros(B, T, 1, 0).double()
        keep = torch.ones(B, T, 1).double()
    n = x * r[..., None] * ww
    val, size = turn(n, c, sn, pairs)
    rel = (0 if norm == "none" else D + 20) * U
    out = dict(out=(val * keep[..., None], (rel + (3 * U if c.shape[-1] else 0)) * size * keep[..., None]),
               r=(r * keep, er * keep))
    if go is None:
        return out
    go = go.double()
    if norm != "none":
        r = r32.double()
    g, size = turn(go, c, sn, pairs, back=True)
    eg = 3 * U * size if c.shape[-1] else 0 * size
    xh = x * r[..., None]
    if norm == "none":
        out["dx"] = (g * keep[..., None], eg * keep[..., None])
        return out
    gw, egw = g * ww, (eg + U * g.abs()) * ww.abs()
    dot = s * (gw * xh).sum(-1, keepdim=True)
    edot = s * ((egw + (D + 16) * U * gw.abs()) * xh.abs()).sum(-1, keepdim=True)
    dx = r[..., None] * (gw - xh * dot)
    edx = r[..., None] * (egw + xh.abs() * edot + 6 * U * (gw.abs() + (xh * dot).abs()))
    rows = (B * T * H + 16) * U
    k4 = keep[..., None]
    out.update(dx=(dx * k4, edx * k4), dw=((g * xh * k4).sum((0, 1, 2)),
                                           (((eg + (rows + 3 * U) * g.abs()) * xh.abs()) * k4).sum((0, 1, 2))))
    return out
