"""Measured cases of the operators around a recurrent layer: the short causal convolution in front of
it, the selective state space scan (a recurrence whose decays are inputs, one for each channel and
state), each for prompts, training and single tokens, and the norm of queries and keys for each
head with the position rotation.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes what
a program holds before the call, ``run()`` is one pass (plain torch where ``own`` is false, the
package's calls where it is true), ``exact()`` the same outputs in 64 bits.
"""
import math

import torch

own = False

SEGMENT = 64        # tokens per segment of the plain scan


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the first words of a chat on a small fp32 model: latency of one short call
        dict(name="scan_short_f32", op="scan", B=1, T=77, C=256, G=1, N=16, io="f32", z=False,
             state=False),
        # one long document read as a prompt (twice the benchmark's 16 heads of 128 channels)
        dict(name="scan_long", op="scan", B=1, T=16384, C=4096, G=1, N=16, io="bf16", z=True,
             state=False),
        # a batch of prompts continued from saved states
        dict(name="scan_batch", op="scan", B=16, T=1021, C=2048, G=1, N=16, io="bf16", z=True,
             state=True),
        # the scan's gradient in a training step
        dict(name="scan_grad", op="scan_grad", B=4, T=2047, C=2048, G=1, N=16, io="bf16", z=True,
             state=False),
        # a training step in fp32 with four groups of input and output vectors, carried states on
        # both sides
        dict(name="scan_grad_groups_f32", op="scan_grad", B=2, T=501, C=1024, G=4, N=32, io="f32",
             z=False, state=True),
        # a server's decode step: 256 places of which a few are empty, states anywhere in the pool
        dict(name="scan_step", op="scan_step", R=256, P=288, C=4096, G=1, N=16, io="bf16", z=True),
        # the convolution in front of the long document's scan
        dict(name="conv_long", op="conv", B=1, T=16384, C=4096, W=4, io="bf16", act="silu",
             state=False),
        # its gradient in a training step on sequences that continue earlier ones
        dict(name="conv_grad", op="conv_grad", B=8, T=2047, C=2048, W=4, io="bf16", act="silu",
             state=True),
        # one user's next token
        dict(name="conv_step_one", op="conv_step", R=1, P=8, C=4096, W=4, io="bf16", act="silu"),
        # queries and keys of a long prompt (the benchmark's heads, keys shared by four each)
        dict(name="qk_long", op="qk", B=1, T=16384, Hq=16, Hk=4, D=128, rot=128, pairs=False,
             norm="rms", io="bf16", table=16384),
        # their gradient in a training step, half of each head's channels rotated, in pairs
        dict(name="qk_grad", op="qk_grad", B=8, T=1023, Hq=16, Hk=16, D=64, rot=32, pairs=True,
             norm="rms", io="bf16", table=1024),
        # one token for each of 64 rows at positions of their own, far into a long context
        dict(name="qk_step", op="qk", B=64, T=1, Hq=16, Hk=4, D=128, rot=128, pairs=False,
             norm="rms", io="bf16", table=131072),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_grad", "scan_grad", "scan_step", "conv", "conv_grad",
                     "conv_step", "qk", "qk_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("scan", "scan_grad", "scan_step"):
        N = rng.choice([4, 8, 16, 16, 16, 16, 24, 32, 64])
        G = rng.choice([1, 1, 1, 2, 4, 8])
        C = G * _log_int(rng, 8, 4096 // G)
        if op == "scan_step":
            R = _log_int(rng, 1, max(1, min(512, (1 << 24) // (C * N))))
            return dict(op=op, R=R, P=R + 1 + rng.randrange(1 + R // 4), C=C, G=G, N=N, io=io,
                        z=rng.random() < 0.7)
        most = (1 << (30 if op == "scan" else 28)) // (C * N)
        T = _log_int(rng, 1, min(16384, most))
        B = _log_int(rng, 1, max(1, min(16, most // T)))
        return dict(op=op, B=B, T=T, C=C, G=G, N=N, io=io, z=rng.random() < 0.7,
                    state=rng.random() < 0.5)
    if op in ("conv", "conv_grad", "conv_step"):
        C = _log_int(rng, 16, 8192)
        if rng.random() < 0.7:
            C = max(8, C // 8 * 8)
        case = dict(op=op, C=C, W=rng.choice([2, 3, 4, 4, 4, 5, 8]), io=io,
                    act=rng.choice(["none", "silu", "silu"]))
        if op == "conv_step":
            R = _log_int(rng, 1, 512)
            return dict(case, R=R, P=R + 1 + rng.randrange(1 + R // 4))
        most = (1 << (26 if op == "conv" else 25)) // C
        T = _log_int(rng, 1, min(16384, most))
        B = _log_int(rng, 1, max(1, min(16, most // T)))
        return dict(case, B=B, T=T, state=rng.random() < 0.5)
    D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 4])
    most = (1 << (25 if op == "qk" else 24)) // ((Hq + Hk) * D)
    T = _log_int(rng, 1, min(16384, most))
    B = _log_int(rng, 1, max(1, min(16, most // T)))
    return dict(op=op, B=B, T=T, Hq=Hq, Hk=Hk, D=D, rot=rng.choice([0, D // 2, D, D]),
                pairs=rng.random() < 0.3, norm=rng.choice(["rms", "rms", "l2", "none"]), io=io,
                table=T + rng.choice([0, 1, 5000]))


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    dt = _dtype(case)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    def slots(R, P):
        s = torch.randperm(P, generator=gen, device="cuda")[:R].to(torch.int32)
        if R > 16:      # places without a sequence
            s[torch.randperm(R, generator=gen, device="cuda")[: R // 16]] = -1
        return s

    op = case["op"]
    if op in ("scan", "scan_grad", "scan_step"):
        C, G, N = case["C"], case["G"], case["N"]
        lead = (case["R"],) if op == "scan_step" else (case["B"], case["T"])
        st = dict(case=case, u=randn(*lead, C, dtype=dt), dt=randn(*lead, C, dtype=dt, std=0.5))
        # B and C are slices of one projection, behind the low-rank part of the step sizes
        rank = max(1, C // 16)
        proj = randn(*lead, rank + 2 * G * N, dtype=dt)
        st["Bm"] = proj[..., rank:rank + G * N].unflatten(-1, (G, N))
        st["Cm"] = proj[..., rank + G * N:].unflatten(-1, (G, N))
        st["z"] = randn(*lead, 2 * C, dtype=dt)[..., C:] if case["z"] else None
        # rates 1 .. N; step sizes of 0.001 to 0.1: memories from a token to a thousand
        rate = torch.arange(1, N + 1, device="cuda", dtype=torch.float32)
        st["A"] = -(rate * torch.exp(0.1 * randn(C, N)))
        step = torch.exp(torch.rand(C, generator=gen, device="cuda") * math.log(100.0) + math.log(1e-3))
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["D"] = 1 + 0.1 * randn(C)
        if op == "scan_step":
            st["S"] = randn(case["P"], C, N)
            st["slots"] = slots(case["R"], case["P"])
            return st
        st["h0"] = randn(case["B"], C, N) if case["state"] else None
        if op == "scan_grad":
            st["do"] = randn(*lead, C, dtype=dt)
            st["dhT"] = randn(case["B"], C, N) if case["state"] else None
        return st
    if op in ("conv", "conv_grad", "conv_step"):
        C, W = case["C"], case["W"]
        lead = (case["R"],) if op == "conv_step" else (case["B"], case["T"])
        # the first half of a projection of twice the width
        st = dict(case=case, x=randn(*lead, 2 * C, dtype=dt)[..., :C], w=randn(C, W, std=W ** -0.5),
                  bias=randn(C, std=0.1))
        if op == "conv_step":
            st["S"] = randn(case["P"], W - 1, C, dtype=dt)
            st["slots"] = slots(case["R"], case["P"])
            return st
        st["s0"] = randn(case["B"], W - 1, C, dtype=dt) if case["state"] else None
        if op == "conv_grad":
            st["dy"] = randn(*lead, C, dtype=dt)
            st["dsT"] = randn(case["B"], W - 1, C, dtype=dt) if case["state"] else None
        return st
    B, T, Hq, Hk, D, rot = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "rot"))
    # slices of one projection of queries, keys and values
    qkv = randn(B, T, (Hq + 2 * Hk) * D, dtype=dt)
    q, k, _ = qkv.split([Hq * D, Hk * D, Hk * D], dim=-1)
    st = dict(case=case, q=q.unflatten(-1, (Hq, D)), k=k.unflatten(-1, (Hk, D)), eps=1e-6, wq=None,
              wk=None, cos=None, sin=None, positions=None)
    if case["norm"] == "rms":
        st["wq"], st["wk"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
    if rot:
        P = case["table"]
        freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = torch.cos(angle).float(), torch.sin(angle).float()
        start = torch.randint(0, P - T + 1, (B, 1), generator=gen, device="cuda")
        st["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
    if op == "qk_grad":
        st["dqo"], st["dko"] = randn(B, T, Hq, D, dtype=dt), randn(B, T, Hk, D, dtype=dt)
        c = 1.0 / D if case["norm"] == "rms" else 1.0
        for n in ("q", "k"):
            r = (c * st[n].float().square().sum(-1) + st["eps"]).rsqrt()
            st["r" + n] = None if case["norm"] == "none" else r
    return st


# ---------------------------------------------------------------- plain forms
def _silu(x):
    return x / (1 + torch.exp(-x))


def _silu_grad(x):
    s = 1 / (1 + torch.exp(-x))
    return s * (1 + x * (1 - s))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _wide(x, C):
    """[..., G, N] -> float [..., C, N], channel c of the result reading group c / (C / G)."""
    return x.float().repeat_interleave(C // x.shape[-2], -2)


def _scan(a, b, h0):
    """All h_t = a_t h_{t-1} + b_t of [B, T, C, N]: segments from zero in lockstep, then the state
    that each starts from."""
    B, T = a.shape[:2]
    n = -(-T // SEGMENT)
    pad = n * SEGMENT - T
    if pad:
        a = torch.cat((a, torch.ones_like(a[:, :1]).expand(-1, pad, -1, -1)), 1)
        b = torch.cat((b, torch.zeros_like(b[:, :1]).expand(-1, pad, -1, -1)), 1)
    a, b = a.unflatten(1, (n, SEGMENT)), b.unflatten(1, (n, SEGMENT))
    h, prod = torch.empty_like(a), torch.empty_like(a)
    s, p = b[:, :, 0], a[:, :, 0]
    h[:, :, 0], prod[:, :, 0] = s, p
    for j in range(1, SEGMENT):
        s, p = a[:, :, j] * s + b[:, :, j], p * a[:, :, j]
        h[:, :, j], prod[:, :, j] = s, p
    start = h0
    for i in range(n):
        h[:, i] += prod[:, i] * start[:, None]
        start = h[:, i, -1]
    return h.flatten(1, 2)[:, :T]


def _scan_inputs(st):
    """Step sizes, decays and inputs of the recurrence, and wide C."""
    c = st["case"]
    delta = _softplus(st["dt"].float() + st["dt_bias"])
    a = torch.exp(delta[..., None] * st["A"])
    Bw, Cw = _wide(st["Bm"], c["C"]), _wide(st["Cm"], c["C"])
    return delta, a, (delta * st["u"].float())[..., None] * Bw, Bw, Cw


def _zero_state(c):
    return torch.zeros(c["B"], c["C"], c["N"], device="cuda")


def _plain_scan(st):
    c = st["case"]
    _, a, b, _, Cw = _scan_inputs(st)
    h = _scan(a, b, _zero_state(c) if st["h0"] is None else st["h0"])
    o = (Cw * h).sum(-1) + st["D"] * st["u"].float()
    if st["z"] is not None:
        o = o * _silu(st["z"].float())
    return o.to(st["u"].dtype), h[:, -1].contiguous()


def _plain_scan_grad(st):
    c = st["case"]
    C, G, dt = c["C"], c["G"], st["u"].dtype
    delta, a, b, Bw, Cw = _scan_inputs(st)
    h0 = _zero_state(c) if st["h0"] is None else st["h0"]
    h = _scan(a, b, h0)
    u, do = st["u"].float(), st["do"].float()
    dy, dz = do, None
    if st["z"] is not None:
        z = st["z"].float()
        dy = do * _silu(z)
        dz = (do * ((Cw * h).sum(-1) + st["D"] * u) * _silu_grad(z)).to(dt)
    # gradient of the state: g_t = C_t dy_t + a_{t+1} g_{t+1}, the last one with dhT
    src = Cw * dy[..., None]
    if st["dhT"] is not None:
        src[:, -1] += st["dhT"]
    after = torch.cat((a[:, 1:], torch.zeros_like(a[:, :1])), 1)
    g = _scan(after.flip(1), src.flip(1), _zero_state(c)).flip(1)
    before = torch.cat((h0[:, None], h[:, :-1]), 1)
    ga = g * before * a                                    # gradient of delta A
    gB = (g * Bw).sum(-1)
    ddelta = (ga * st["A"]).sum(-1) + gB * u
    du = gB * delta + st["D"] * dy
    raw = st["dt"].float() + st["dt_bias"]
    ddt = ddelta / (1 + torch.exp(-raw))
    dA = (ga * delta[..., None]).sum((0, 1))
    share = lambda t: t.unflatten(2, (G, C // G)).sum(3).to(dt)      # noqa: E731
    dB = share(g * (delta * u)[..., None])
    dC = share(h * dy[..., None])
    out = [du.to(dt), ddt.to(dt), dA, dB, dC, (dy * u).sum((0, 1)), ddt.sum((0, 1))]
    if dz is not None:
        out.append(dz)
    if st["h0"] is not None:
        out.append(a[:, 0] * g[:, 0])
    return out


def _plain_scan_step(st):
    c = st["case"]
    some = st["slots"] >= 0
    at = st["slots"][some].long()
    _, a, b, _, Cw = _scan_inputs(st)
    S = a[some] * st["S"][at] + b[some]
    st["S"][at] = S
    y = (Cw[some] * S).sum(-1) + st["D"] * st["u"][some].float()
    if st["z"] is not None:
        y = y * _silu(st["z"][some].float())
    o = torch.zeros(c["R"], c["C"], device="cuda")
    o[some] = y
    return o.to(st["u"].dtype), st["S"]


def _behind(x, s0, W):
    """float [B, W - 1 + T, C]: the inputs with those before the first one."""
    if s0 is None:
        s0 = torch.zeros(x.shape[0], W - 1, x.shape[2], device="cuda")
    return torch.cat((s0.float(), x.float()), 1)


def _conv_sum(xs, w, bias, T):
    u = bias + w[:, 0] * xs[:, :T]
    for j in range(1, w.shape[1]):
        u = u + w[:, j] * xs[:, j:j + T]
    return u


def _plain_conv(st):
    c = st["case"]
    x, W, T = st["x"], c["W"], c["T"]
    xs = _behind(x, st["s0"], W)
    u = _conv_sum(xs, st["w"], st["bias"], T)
    y = _silu(u) if c["act"] == "silu" else u
    return y.to(x.dtype), xs[:, T:].to(x.dtype)


def _plain_conv_grad(st):
    c = st["case"]
    x, W, T, dt = st["x"], c["W"], c["T"], st["x"].dtype
    xs = _behind(x, st["s0"], W)
    du = st["dy"].float()
    if c["act"] == "silu":
        du = du * _silu_grad(_conv_sum(xs, st["w"], st["bias"], T))
    dxs = torch.zeros_like(xs)
    if st["dsT"] is not None:
        dxs[:, T:] += st["dsT"].float()
    for j in range(W):
        dxs[:, j:j + T] += st["w"][:, j] * du
    dw = torch.stack([(du * xs[:, j:j + T]).sum((0, 1)) for j in range(W)], 1)
    out = [dxs[:, W - 1:].to(dt), dw, du.sum((0, 1))]
    return out + ([dxs[:, :W - 1].to(dt)] if st["s0"] is not None else [])


def _plain_conv_step(st):
    c = st["case"]
    some = st["slots"] >= 0
    at = st["slots"][some].long()
    xs = torch.cat((st["S"][at], st["x"][some][:, None]), 1)          # [rows, W, C]
    st["S"][at] = xs[:, 1:]
    u = (xs.float() * st["w"].t()).sum(1) + st["bias"]
    y = torch.zeros(c["R"], c["C"], device="cuda")
    y[some] = _silu(u) if c["act"] == "silu" else u
    return y.to(st["x"].dtype), st["S"]


def _turn(st, n, back=False):
    """The rotation of the first ``rot`` channels of float n [B, T, H, D] (its transpose: back)."""
    c = st["case"]
    rot = c["rot"]
    if not rot:
        return n
    at = st["positions"].long()
    cos, sin = st["cos"][at][:, :, None], st["sin"][at][:, :, None]
    if back:
        sin = -sin
    a, b = ((n[..., 0:rot:2], n[..., 1:rot:2]) if c["pairs"] else
            (n[..., :rot // 2], n[..., rot // 2:rot]))
    x, y = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((x, y), -1).flatten(-2) if c["pairs"] else torch.cat((x, y), -1)
    return torch.cat((r, n[..., rot:]), -1)


def _norm_scale(c):
    return 1.0 / c["D"] if c["norm"] == "rms" else 1.0


def _plain_qk(st):
    c = st["case"]
    outs, stats = [], []
    for name in ("q", "k"):
        x, w = st[name].float(), st["w" + name]
        if c["norm"] != "none":
            r = (_norm_scale(c) * x.square().sum(-1) + st["eps"]).rsqrt()
            x = x * r[..., None]
            stats.append(r)
        if w is not None:
            x = x * w
        outs.append(_turn(st, x).to(st[name].dtype))
    return outs + stats


def _plain_qk_grad(st):
    c = st["case"]
    outs, sums = [], []
    for name in ("q", "k"):
        x, w, r = st[name].float(), st["w" + name], st["r" + name]
        g = _turn(st, st["d" + name + "o"].float(), True)
        if w is not None:
            sums.append((g * x * r[..., None]).sum((0, 1, 2)))
            g = g * w
        if r is not None:
            r = r[..., None]
            g = r * (g - x * (_norm_scale(c) * r * r * (g * x).sum(-1, keepdim=True)))
        outs.append(g.to(st[name].dtype))
    return outs + sums


_PLAIN = dict(scan=_plain_scan, scan_grad=_plain_scan_grad, scan_step=_plain_scan_step,
              conv=_plain_conv, conv_grad=_plain_conv_grad, conv_step=_plain_conv_step,
              qk=_plain_qk, qk_grad=_plain_qk_grad)


def _own(st):
    import chunkwise_recurrent_prefill_gb300 as pkg
    c = st["case"]
    op = c["op"]
    if op == "scan":
        return pkg.ssm_fwd(st["u"], st["dt"], st["A"], st["Bm"], st["Cm"], D=st["D"], z=st["z"],
                           dt_bias=st["dt_bias"], h0=st["h0"], softplus=True, return_state=True)
    if op == "scan_grad":
        du, ddt, dA, dB, dC, dD, dz, dbias, dh0 = pkg.ssm_bwd(
            st["do"], st["u"], st["dt"], st["A"], st["Bm"], st["Cm"], D=st["D"], z=st["z"],
            dt_bias=st["dt_bias"], h0=st["h0"], dhT=st["dhT"], softplus=True)
        return [du, ddt, dA, dB, dC, dD, dbias] + [t for t in (dz, dh0) if t is not None]
    if op == "scan_step":
        o = pkg.ssm_step(st["u"], st["dt"], st["A"], st["Bm"], st["Cm"], st["S"], st["slots"],
                         D=st["D"], z=st["z"], dt_bias=st["dt_bias"], softplus=True)
        return o, st["S"]
    if op == "conv":
        return pkg.conv_fwd(st["x"], st["w"], st["bias"], st["s0"], act=c["act"], return_state=True)
    if op == "conv_grad":
        dx, dw, db, ds0 = pkg.conv_bwd(st["dy"], st["x"], st["w"], st["bias"], st["s0"], st["dsT"],
                                       act=c["act"])
        return [dx, dw, db] + ([ds0] if ds0 is not None else [])
    if op == "conv_step":
        return pkg.conv_step(st["x"], st["w"], st["S"], st["slots"], st["bias"], act=c["act"]), st["S"]
    how = dict(norm=c["norm"], layout="pairs" if c["pairs"] else "halves")
    if op == "qk":
        qo, ko, rq, rk = pkg.qk_norm_fwd(st["q"], st["k"], st["wq"], st["wk"], cos=st["cos"],
                                         sin=st["sin"], positions=st["positions"], eps=st["eps"], **how)
        return [qo, ko] + [t for t in (rq, rk) if t is not None]
    dq, dk, dwq, dwk = pkg.qk_norm_bwd(st["dqo"], st["dko"], st["q"], st["k"], st["rq"], st["rk"],
                                       st["wq"], st["wk"], cos=st["cos"], sin=st["sin"],
                                       positions=st["positions"], **how)
    return [dq, dk] + [t for t in (dwq, dwk) if t is not None]


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _exact_scan(case, st):
    """Token by token."""
    op, C, G = case["op"], case["C"], case["G"]
    f = {n: (None if st.get(n) is None else st[n].double())
         for n in ("u", "dt", "Bm", "Cm", "z", "A", "D", "dt_bias", "S", "h0", "do", "dhT")}
    A, D = f["A"], f["D"]
    group = torch.arange(C, device="cuda") // (C // G)
    raw = f["dt"] + f["dt_bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    du64 = delta * f["u"]
    if op == "scan_step":
        o = torch.zeros_like(f["u"])
        for r, s in enumerate(st["slots"].tolist()):
            if s < 0:
                continue
            S = torch.exp(delta[r][:, None] * A) * f["S"][s] + du64[r][:, None] * f["Bm"][r][group]
            f["S"][s] = S
            y = (f["Cm"][r][group] * S).sum(1) + D * f["u"][r]
            o[r] = y if f["z"] is None else y * f["z"][r] * torch.sigmoid(f["z"][r])
        return o, f["S"]
    B, T, N = case["B"], case["T"], case["N"]
    start = torch.zeros(B, C, N, device="cuda", dtype=torch.float64) if f["h0"] is None else f["h0"]
    keep = op == "scan_grad"
    h, hs, y = start, [], torch.empty_like(f["u"])
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * A) * h + du64[:, t, :, None] * f["Bm"][:, t][:, group]
        y[:, t] = (f["Cm"][:, t][:, group] * h).sum(2)
        if keep:
            hs.append(h)
    y += D * f["u"]
    gate = None if f["z"] is None else f["z"] * torch.sigmoid(f["z"])
    if not keep:
        return (y if gate is None else y * gate), h
    dy, out_z = f["do"], []
    if gate is not None:
        s = torch.sigmoid(f["z"])
        out_z = [f["do"] * y * (s + f["z"] * s * (1 - s))]
        dy = f["do"] * gate
    g = torch.zeros_like(start) if f["dhT"] is None else f["dhT"].clone()
    dA = torch.zeros_like(A)
    du, ddelta = torch.empty_like(dy), torch.empty_like(dy)
    dB, dC = torch.empty(B, T, G, N, device="cuda").double(), torch.empty(B, T, G, N, device="cuda").double()
    for t in range(T - 1, -1, -1):
        g = g + f["Cm"][:, t][:, group] * dy[:, t, :, None]
        a = torch.exp(delta[:, t, :, None] * A)
        w = g * a * (hs[t - 1] if t else start)
        gb = (g * f["Bm"][:, t][:, group]).sum(2)
        ddelta[:, t] = (w * A).sum(2) + gb * f["u"][:, t]
        du[:, t] = gb * delta[:, t] + D * dy[:, t]
        dA += (w * delta[:, t, :, None]).sum(0)
        dB[:, t] = (g * du64[:, t, :, None]).unflatten(1, (G, C // G)).sum(2)
        dC[:, t] = (hs[t] * dy[:, t, :, None]).unflatten(1, (G, C // G)).sum(2)
        g = a * g
    ddt = ddelta * torch.sigmoid(raw)
    out = [du, ddt, dA, dB, dC, (dy * f["u"]).sum((0, 1)), ddt.sum((0, 1))] + out_z
    return out + ([g] if f["h0"] is not None else [])


def _exact_conv(case, st):
    op, C, W = case["op"], case["C"], case["W"]
    f = torch.nn.functional.silu if case["act"] == "silu" else (lambda t: t)
    x, w, b = (st[n].double() for n in ("x", "w", "bias"))
    if op == "conv_step":
        S, y = st["S"].double(), torch.zeros_like(x)
        for r, s in enumerate(st["slots"].tolist()):
            if s >= 0:
                line = torch.cat((S[s], x[r:r + 1]))
                y[r] = f(torch.einsum("wc,cw->c", line, w) + b)
                S[s] = line[1:]
        return y, S
    B, T = case["B"], case["T"]
    s0 = torch.zeros(B, W - 1, C, device="cuda").double() if st["s0"] is None else st["s0"].double()
    leaves = [t.requires_grad_() for t in (x, w, b, s0)]
    line = torch.cat((s0, x), 1)
    y = f(torch.einsum("btcw,cw->btc", line.unfold(1, W, 1), w) + b)
    sT = line[:, T:]
    if op == "conv":
        return y.detach(), sT.detach()
    dsT = torch.zeros_like(s0) if st["dsT"] is None else st["dsT"].double()
    grads = torch.autograd.grad([y, sT], leaves, [st["dy"].double(), dsT])
    return list(grads if st["s0"] is not None else grads[:3])


def _exact_qk(case, st):
    D, rot = case["D"], case["rot"]
    # the rotation as a complex product
    if rot:
        at = st["positions"].long()
        turn = torch.complex(st["cos"].double(), st["sin"].double())[at][:, :, None]
        i = torch.arange(rot, device="cuda")
        first = i[0::2] if case["pairs"] else i[:rot // 2]
        second = i[1::2] if case["pairs"] else i[rot // 2:]
    outs, stats, sums = [], [], []
    for name in ("q", "k"):
        x = st[name].double().requires_grad_()
        w = None if st["w" + name] is None else st["w" + name].double().requires_grad_()
        n = x
        if case["norm"] != "none":
            ss = (x * x).mean(-1) if case["norm"] == "rms" else (x * x).sum(-1)
            r = 1 / torch.sqrt(ss + st["eps"])
            stats.append(r.detach())
            if case["op"] == "qk_grad":       # the stored factor is an input of the gradient
                r = r * (st["r" + name].double() / r).detach()
                # ... whose own derivative is taken at the stored value
                r0 = st["r" + name].double()
                r = r0 + (-0.5 * r0 ** 3 * ss - (-0.5 * r0 ** 3 * ss).detach())
            n = x * r[..., None]
        if w is not None:
            n = n * w
        if rot:
            v = torch.complex(n[..., first], n[..., second]) * turn
            cols = torch.cat((v.real, v.imag), -1)
            order = torch.empty(rot, dtype=torch.long, device="cuda")
            order[torch.cat((first, second))] = torch.arange(rot, device="cuda")
            n = torch.cat((cols[..., order], n[..., rot:]), -1)
        if case["op"] == "qk":
            outs.append(n.detach())
            continue
        grads = torch.autograd.grad(n, [x] + ([w] if w is not None else []), st["d" + name + "o"].double())
        outs.append(grads[0])
        sums += list(grads[1:])
    return outs + (stats if case["op"] == "qk" else sums)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["op"].split("_")[0]
    return dict(scan=_exact_scan, conv=_exact_conv, qk=_exact_qk)[kind](case, st)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    es = 2 if case["io"] == "bf16" else 4
    if op in ("scan", "scan_grad", "scan_step"):
        C, G, N = case["C"], case["G"], case["N"]
        cn, params = C * N, C * N * 4 + C * 8
        if op == "scan_step":
            R = case["R"]
            rows = R - (R // 16 if R > 16 else 0)
            return dict(bytes=params + rows * (es * ((4 if case["z"] else 3) * C + 2 * G * N) + 8 * cn),
                        flops=7 * rows * cn)
        tokens = case["B"] * case["T"]
        states = case["B"] * cn * 4
        row = (4 if case["z"] else 3) * C + 2 * G * N
        if op == "scan":
            return dict(bytes=params + tokens * es * row + states * (2 if case["state"] else 1),
                        flops=7 * tokens * cn)
        # read: u, dt, do (z), B, C; written: du, ddt (dz), dB, dC
        row = (7 if case["z"] else 5) * C + 4 * G * N
        return dict(bytes=2 * params + tokens * es * row + states * (3 if case["state"] else 0),
                    flops=21 * tokens * cn)
    if op in ("conv", "conv_grad", "conv_step"):
        C, W = case["C"], case["W"]
        params = C * (W + 1) * 4
        if op == "conv_step":
            R = case["R"]
            rows = R - (R // 16 if R > 16 else 0)
            return dict(bytes=params + rows * es * C * (2 + 2 * (W - 1)), flops=(2 * W + 5) * rows * C)
        n, state = case["B"] * case["T"] * C, case["B"] * (W - 1) * C * es
        if op == "conv":
            return dict(bytes=params + 2 * n * es + state * (2 if case["state"] else 1),
                        flops=(2 * W + 5) * n)
        return dict(bytes=2 * params + 3 * n * es + (3 * state if case["state"] else 0),
                    flops=(6 * W + 10) * n)
    tokens, heads, D = case["B"] * case["T"], case["Hq"] + case["Hk"], case["D"]
    n = tokens * heads * D
    # the angles' table once for each row of it that a position names
    table = min(tokens, case["table"]) * case["rot"] * 4 + (tokens * 4 if case["rot"] else 0)
    stats = 0 if case["norm"] == "none" else tokens * heads * 4
    if op == "qk":
        return dict(bytes=2 * n * es + table + stats, flops=8 * n)
    return dict(bytes=3 * n * es + table + stats, flops=16 * n)
