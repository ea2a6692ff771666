"""Measured cases of the decay-attention operators: attention with one decay per head (prompts,
training, single tokens), the group norm that follows it, and the pages of the state pool.

``listed()`` names the cases, ``draw()`` gives more of the same ranges, ``prepare()`` makes what
a program holds before the call, ``run()`` is one pass (plain torch where ``own`` is false, the
package's calls where it is true), ``exact()`` the same outputs in 64 bits.
"""
import math

import torch

own = False

CHUNK = 64          # tokens per chunk of the plain form


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the first words of a chat on a small fp32 model: latency of one short call
        dict(name="prompt_short_f32", op="prompt", B=1, T=77, H=4, Hq=4, Hk=4, Hv=4, Dk=64, Dv=64,
             io="f32", decay="slopes", state=False),
        # one long document read as a prompt (the benchmark's shape)
        dict(name="prompt_long", op="prompt", B=1, T=16384, H=16, Hq=16, Hk=16, Hv=16, Dk=128,
             Dv=128, io="bf16", decay="slow", state=False),
        # a batch of prompts continued from saved states, keys and values shared by four heads each
        dict(name="prompt_batch_shared", op="prompt", B=16, T=2501, H=16, Hq=16, Hk=4, Hv=4,
             Dk=128, Dv=128, io="bf16", decay="slopes", state=True),
        # the attention's gradient in a training step on long documents
        dict(name="grad_long", op="grad", B=1, T=16384, H=16, Hq=16, Hk=16, Hv=16, Dk=128, Dv=128,
             io="bf16", decay="slow", state=False),
        # a training step on a batch of shorter texts, queries and keys shared by four heads each,
        # carried states on both sides, head dims of 64
        dict(name="grad_batch_shared", op="grad", B=8, T=1023, H=16, Hq=4, Hk=4, Hv=16, Dk=64,
             Dv=64, io="bf16", decay="slopes", state=True),
        # one user's next token
        dict(name="step_one", op="step", R=1, P=8, H=16, Hq=16, Hk=16, Hv=16, Dk=128, Dv=128,
             io="bf16", decay="slopes"),
        # a server's decode step: 256 places of which a few are empty, states anywhere in the pool
        dict(name="step_batch", op="step", R=256, P=288, H=16, Hq=16, Hk=4, Hv=4, Dk=128, Dv=128,
             io="bf16", decay="slow"),
        # the norm over each head's output of a long prompt, times the gate branch
        dict(name="norm_tokens", op="norm", N=16384, L=1, C=2048, G=16, io="bf16", act="silu",
             gate=True),
        # its gradient in a training step
        dict(name="norm_tokens_grad", op="norm_grad", N=8191, L=1, C=2048, G=16, io="bf16",
             act="silu", gate=True),
        # the norm over whole feature maps, channels last, activation behind it
        dict(name="norm_maps", op="norm", N=3, L=4095, C=512, G=32, io="bf16", act="silu",
             gate=False),
        # 64 beams or samples split off from running sequences
        dict(name="fork_beams", op="fork", P=256, R=160, M=1, n=64, page=262144),
        # a pool of small pages (one for each of 8 layers) closed up after half the rows ended
        dict(name="compact_rows", op="compact", P=640, R=64, M=8, page=65536),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _divisor(rng, h):
    return rng.choice([d for d in range(1, h + 1) if h % d == 0 and d * 8 >= h])


def draw(rng):
    op = rng.choice(["prompt", "prompt", "grad", "grad", "step", "norm", "norm_grad", "fork",
                     "compact"])
    if op in ("prompt", "grad"):
        io = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = (1 << 19) // (2 if op == "grad" else 1) if io == "bf16" else 1 << 15
        H = rng.choice([1, 2, 4, 6, 8, 12, 16, 24, 32])
        T = _log_int(rng, 1, min(16384, most // H))
        B = _log_int(rng, 1, max(1, min(16, most // (H * T))))
        return dict(op=op, B=B, T=T, H=H, Hq=_divisor(rng, H), Hk=_divisor(rng, H),
                    Hv=_divisor(rng, H), Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128]), io=io,
                    decay=rng.choice(["slopes", "slow"]), state=rng.random() < 0.5)
    if op == "step":
        H = rng.choice([1, 2, 4, 8, 12, 16, 32])
        R = _log_int(rng, 1, 4096 // H)
        return dict(op=op, R=R, P=R + 1 + rng.randrange(1 + R // 4), H=H, Hq=_divisor(rng, H),
                    Hk=_divisor(rng, H), Hv=_divisor(rng, H), Dk=rng.choice([64, 128]),
                    Dv=rng.choice([64, 128]), io=rng.choice(["bf16", "bf16", "f32"]),
                    decay=rng.choice(["slopes", "slow"]))
    if op in ("norm", "norm_grad"):
        G = rng.choice([1, 2, 4, 8, 16, 32])
        C = G * rng.choice([8, 16, 24, 40, 64, 96, 128])
        most = (1 << 24) // C
        if rng.random() < 0.5:
            N, L = _log_int(rng, 1, min(most, 16384)), 1
        else:
            L = _log_int(rng, 2, min(most, 16384))
            N = _log_int(rng, 1, max(1, min(8, most // L)))
        return dict(op=op, N=N, L=L, C=C, G=G, io=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "silu", "gelu"]), gate=rng.random() < 0.5)
    page = 16 * _log_int(rng, 64, 16384)
    M = rng.choice([1, 1, 2, 5, 8])
    R = _log_int(rng, 2, 200 if M < 5 else 64)
    P = 2 * R * M + rng.randrange(8)
    while P * page > 1 << 26:
        page = 16 * max(4, page // 32)
    if op == "fork":
        return dict(op=op, P=P, R=R, M=M, n=rng.randrange(1, max(2, R // 2)), page=page)
    return dict(op=op, P=P, R=R, M=M, page=page)


# ---------------------------------------------------------------- inputs
def _dtype(case):
    return torch.bfloat16 if case["io"] == "bf16" else torch.float32


def _decays(case):
    H = case["H"]
    h = torch.arange(1, H + 1, dtype=torch.float64)
    if case["decay"] == "slopes":              # from 0.7 a token down to 1/256
        g = -torch.exp2(-8.0 * h / H) if H > 1 else -torch.exp2(-8.0 * h / 2)
    else:                                      # 1 - 2^-5 ... 1 - 2^-10: memories of 32 to 1024 tokens
        g = torch.log1p(-torch.exp2(-5.0 - 5.0 * (h - 1) / max(H - 1, 1)))
    return g.float().cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    op = case["op"]
    if op in ("prompt", "grad", "step"):
        H, Hq, Hk, Hv, Dk, Dv = (case[n] for n in ("H", "Hq", "Hk", "Hv", "Dk", "Dv"))
        lead = (case["R"],) if op == "step" else (case["B"], case["T"])
        # one projection's output, of which q, k and v are slices
        qkv = randn(*lead, Hq * Dk + Hk * Dk + Hv * Dv, dtype=_dtype(case))
        q, k, v = qkv.split([Hq * Dk, Hk * Dk, Hv * Dv], dim=-1)
        st = dict(case=case, q=q.unflatten(-1, (Hq, Dk)), k=k.unflatten(-1, (Hk, Dk)),
                  v=v.unflatten(-1, (Hv, Dv)), decay=_decays(case), scale=float(Dk) ** -0.5)
        if op == "step":
            P, R = case["P"], case["R"]
            st["S"] = randn(P, H, Dk, Dv)
            slots = torch.randperm(P, generator=gen, device="cuda")[:R].to(torch.int32)
            if R > 16:      # places without a sequence
                slots[torch.randperm(R, generator=gen, device="cuda")[: R // 16]] = -1
            st["slots"] = slots
            return st
        B, T = lead
        st["h0"] = randn(B, H, Dk, Dv) if case["state"] else None
        if op == "grad":
            st["do"] = randn(B, T, H, Dv, dtype=_dtype(case))
            st["dhT"] = randn(B, H, Dk, Dv) if case["state"] else None
        return st
    if op in ("norm", "norm_grad"):
        N, L, C, G = (case[n] for n in ("N", "L", "C", "G"))
        dt = _dtype(case)
        x = (randn(N, L, C) * (1 + 0.2 * randn(C)) + 0.3 * randn(C)).to(dt)
        st = dict(case=case, x=x, w=1 + 0.1 * randn(C), b=0.1 * randn(C), eps=1e-5, gate=None)
        if case["gate"]:    # the other half of a projection of twice the width
            st["gate"] = randn(N, L, 2 * C, dtype=dt)[..., C:]
        if op == "norm_grad":
            st["dy"] = randn(N, L, C, dtype=dt)
            xg = x.float().view(N, L, G, C // G)
            mean = xg.mean((1, 3))
            st["mean"] = mean
            st["rstd"] = (xg.var((1, 3), unbiased=False) + st["eps"]).rsqrt()
        return st
    # pages
    P, R, M = case["P"], case["R"], case["M"]
    pool = randn(P, case["page"])
    perm = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    rows = torch.randperm(R, generator=gen, device="cuda")
    # the bookkeeping in one buffer: table, free stack, count
    meta = torch.full((R * M + P + 1,), -1, dtype=torch.int32, device="cuda")
    n_live = R - case["n"] if op == "fork" else (R + 1) // 2
    live = n_live * M
    table = meta[: R * M].view(R, M)
    table[rows[:n_live]] = perm[:live].view(n_live, M)
    meta[R * M: R * M + P - live] = perm[live:]
    meta[-1] = P - live
    st = dict(case=case, pool=pool, meta=meta)
    if op == "fork":
        st["parents"] = rows[torch.randint(0, n_live, (case["n"],), generator=gen,
                                           device="cuda")].to(torch.int32)
        st["children"] = rows[n_live:].to(torch.int32)
    return st


# ---------------------------------------------------------------- plain forms
def _heads(x, H):
    """[B, T, h, D] -> float [B, H, T, D], head h of the result reading head h / (H / h)."""
    return x.float().transpose(1, 2).repeat_interleave(H // x.shape[2], 1)


def _powers(decay, n):
    e = torch.arange(n, device="cuda", dtype=torch.float32)
    return torch.where(e == 0, 1.0, torch.exp(decay[:, None] * e))      # [H, n]


def _lin(x, y, z, decay, S, reverse):
    """out_i = sum_j l^|i-j| (x_i . y_j) z_j + (state term) over j <= i (j >= i in reverse), and
    the state at the end: the map that the forward and all three gradients are made of. Before
    the first token (after the last, in reverse) the state is S: a token at distance m from it
    reads l^(m+1) S forwards and l^m S in reverse, and adds l^(rest) y z to it."""
    T = x.shape[2]
    if reverse:
        x, y, z = x.flip(2), y.flip(2), z.flip(2)
    outs = []
    N = T // CHUNK
    for C, lo, n in ((CHUNK, 0, N), (T - N * CHUNK, N * CHUNK, 1)):
        if C == 0 or n == 0:
            continue
        xs, ys, zs = (t[:, :, lo:lo + n * C].unflatten(2, (n, C)) for t in (x, y, z))
        pw = _powers(decay, C + 1)
        i = torch.arange(C, device="cuda")
        d = i[:, None] - i[None, :]
        m = torch.where(d >= 0, pw[:, d.clamp(min=0)], 0.0)             # [H, C, C]
        fin = pw[:, :C] if reverse else pw[:, 1:C + 1]                   # state -> output
        fout = pw[:, 1:C + 1].flip(1) if reverse else pw[:, :C].flip(1)  # token -> state
        intra = (xs @ ys.transpose(-1, -2) * m[:, None]) @ zs
        add = ys.transpose(-1, -2) @ (zs * fout[:, None, :, None])
        starts = []
        for c in range(n):
            starts.append(S)
            S = pw[:, C, None, None] * S + add[:, :, c]
        inter = xs @ torch.stack(starts, 2)
        outs.append((intra + fin[:, None, :, None] * inter).flatten(2, 3))
    out = torch.cat(outs, 2)
    return (out.flip(2) if reverse else out), S


def _share(d, h):
    """[B, H, T, D] -> [B, T, h, D]: gradients of the heads that share an input, summed."""
    B, H, T, D = d.shape
    return d.view(B, h, H // h, T, D).sum(2).transpose(1, 2)


def _plain_prompt(st):
    c = st["case"]
    q, k, v = (_heads(st[n], c["H"]) for n in "qkv")
    S = st["h0"] if st["h0"] is not None else torch.zeros(c["B"], c["H"], c["Dk"], c["Dv"],
                                                          device="cuda")
    o, S = _lin(q * st["scale"], k, v, st["decay"], S, False)
    return o.transpose(1, 2).to(st["q"].dtype).contiguous(), S


def _plain_grad(st):
    c = st["case"]
    H, dt = c["H"], st["q"].dtype
    q, k, v = (_heads(st[n], H) for n in "qkv")
    do = _heads(st["do"], H) * st["scale"]
    zero = torch.zeros(c["B"], H, c["Dk"], c["Dv"], device="cuda")
    h0 = st["h0"] if st["h0"] is not None else zero
    dhT = st["dhT"] if st["dhT"] is not None else zero
    dq, _ = _lin(do, v, k, st["decay"], h0.transpose(2, 3), False)
    dk, _ = _lin(v, do, q, st["decay"], dhT.transpose(2, 3), True)
    dv, dh0 = _lin(k, q, do, st["decay"], dhT, True)
    out = [_share(d, c[n]).to(dt).contiguous() for d, n in ((dq, "Hq"), (dk, "Hk"), (dv, "Hv"))]
    return out + ([dh0] if st["h0"] is not None else [])


def _plain_step(st):
    c = st["case"]
    q, k, v = (st[n].float().repeat_interleave(c["H"] // st[n].shape[1], 1) for n in "qkv")
    some = st["slots"] >= 0
    at = st["slots"][some].long()
    S = (st["S"][at] * torch.exp(st["decay"])[:, None, None]
         + k[some][..., :, None] * v[some][..., None, :])
    st["S"][at] = S
    o = torch.zeros(c["R"], c["H"], c["Dv"], device="cuda")
    o[some] = st["scale"] * (q[some][..., None, :] @ S).squeeze(-2)
    return o.to(st["q"].dtype), st["S"]


def _act(u, act):
    if act == "silu":
        return u / (1 + torch.exp(-u))
    if act == "gelu":
        return 0.5 * u * (1 + torch.erf(u * 0.5 ** 0.5))
    return u


def _act_grad(u, act):
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return s * (1 + u * (1 - s))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(u * 0.5 ** 0.5))
                + u * torch.exp(-0.5 * u * u) * (2 * math.pi) ** -0.5)
    return torch.ones_like(u)


def _plain_norm(st):
    c = st["case"]
    N, L, C, G = (c[n] for n in ("N", "L", "C", "G"))
    x = st["x"].float().view(N, L, G, C // G)
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + st["eps"]).rsqrt()
    u = ((x - mean) * rstd).view(N, L, C) * st["w"] + st["b"]
    y = _act(u, c["act"]) if st["gate"] is None else u * _act(st["gate"].float(), c["act"])
    return y.to(st["x"].dtype), mean.view(N, G), rstd.view(N, G)


def _plain_norm_grad(st):
    c = st["case"]
    N, L, C, G = (c[n] for n in ("N", "L", "C", "G"))
    dt = st["x"].dtype
    rstd = st["rstd"].view(N, 1, G, 1)
    xh = ((st["x"].float().view(N, L, G, C // G) - st["mean"].view(N, 1, G, 1)) * rstd)
    xc = xh.view(N, L, C)
    u = xc * st["w"] + st["b"]
    dy = st["dy"].float()
    if st["gate"] is None:
        du, dz = dy * _act_grad(u, c["act"]), None
    else:
        z = st["gate"].float()
        du, dz = dy * _act(z, c["act"]), (dy * u * _act_grad(z, c["act"])).to(dt)
    dxh = (du * st["w"]).view(N, L, G, C // G)
    dx = rstd * (dxh - dxh.mean((1, 3), keepdim=True)
                 - xh * (dxh * xh).mean((1, 3), keepdim=True))
    out = [dx.view(N, L, C).to(dt), (du * xc).sum((0, 1)), du.sum((0, 1))]
    return out + ([dz] if dz is not None else [])


def _meta(st):
    """Views of a fresh copy of the bookkeeping: the whole buffer, table, free stack, count."""
    c = st["case"]
    m = st["meta"].clone()
    n = c["R"] * c["M"]
    return m, m[:n].view(c["R"], c["M"]), m[n:n + c["P"]], m[n + c["P"]:]


def _plain_fork(st):
    meta, table, free, count = _meta(st)
    src = table[st["parents"].long()]                                   # [n, M]
    rank = torch.cumsum((src >= 0).view(-1), 0).view(src.shape) - 1
    new = torch.where(src >= 0, free[(count - 1 - rank).clamp(min=0).long()], -1)
    have = src >= 0
    st["pool"][new[have].long()] = st["pool"][src[have].long()]
    table[st["children"].long()] = new
    count -= have.sum().to(torch.int32)
    return st["pool"], meta


def _plain_compact(st):
    meta, table, free, count = _meta(st)
    P = free.numel()
    live = torch.zeros(P, dtype=torch.bool, device="cuda")
    live[table[table >= 0].long()] = True
    page = torch.arange(P, device="cuda")
    n = live.sum()
    src = page[live & (page >= n)]
    dst = page[~live & (page < n)]
    st["pool"][dst] = st["pool"][src]
    to = page.clone()
    to[src] = dst
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    count.copy_(P - n)
    free.copy_(torch.where(page < P - n, P - 1 - page, -1))
    return st["pool"], meta


_PLAIN = dict(prompt=_plain_prompt, grad=_plain_grad, step=_plain_step, norm=_plain_norm,
              norm_grad=_plain_norm_grad, fork=_plain_fork, compact=_plain_compact)


def _own(st):
    import chunkwise_recurrent_prefill_gb300 as pkg
    c = st["case"]
    op = c["op"]
    if op == "prompt":
        return pkg.hda_fwd(st["q"], st["k"], st["v"], st["decay"], st["scale"], st["h0"],
                           return_state=True)
    if op == "grad":
        dq, dk, dv, dh0 = pkg.hda_bwd(st["do"], st["q"], st["k"], st["v"], st["decay"],
                                      st["scale"], st["h0"], st["dhT"])
        return [dq, dk, dv] + ([dh0] if dh0 is not None else [])
    if op == "step":
        o = pkg.hda_step(st["q"], st["k"], st["v"], st["decay"], st["scale"], st["S"],
                         st["slots"])
        return o, st["S"]
    if op == "norm":
        return pkg.group_norm_fwd(st["x"], c["G"], st["w"], st["b"], eps=st["eps"], act=c["act"],
                                  gate=st["gate"])
    if op == "norm_grad":
        dx, dw, db, dz = pkg.group_norm_bwd(st["dy"], st["x"], st["mean"], st["rstd"], c["G"],
                                            st["w"], st["b"], act=c["act"], gate=st["gate"])
        return [dx, dw, db] + ([dz] if dz is not None else [])
    meta, table, free, count = _meta(st)
    if op == "fork":
        pkg.pages_fork(st["pool"], table, free, count, st["parents"], st["children"])
    else:
        pkg.pages_compact(st["pool"], table, free, count)
    return st["pool"], meta


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits
def _scan64(x, y, z, lam, S, scale):
    """o_t = scale x_t S_t with S_t = lam S_{t-1} + y_t^T z_t, token by token."""
    out = []
    for t in range(x.shape[1]):
        S = lam * S + y[:, t, :, :, None] * z[:, t, :, None, :]
        out.append((x[:, t, :, None, :] @ S)[:, :, 0] * scale)
    return torch.stack(out, 1), S


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("prompt", "grad", "step"):
        H = case["H"]
        lam = torch.exp(st["decay"].double())[:, None, None]
        q, k, v = (st[n].double() for n in "qkv")
        wide = lambda t: t[..., torch.arange(H, device="cuda") // (H // t.shape[-2]), :]  # noqa: E731
        q, k, v = wide(q), wide(k), wide(v)
        sc = st["scale"]
        if op == "step":
            S, o = st["S"].double(), torch.zeros(case["R"], H, case["Dv"], device="cuda").double()
            for r, s in enumerate(st["slots"].tolist()):
                if s >= 0:
                    S[s] = lam * S[s] + k[r, :, :, None] * v[r, :, None, :]
                    o[r] = sc * (q[r, :, None, :] @ S[s])[:, 0]
            return o, S
        B, T, Dk, Dv = case["B"], case["T"], case["Dk"], case["Dv"]
        zero = torch.zeros(B, H, Dk, Dv, device="cuda", dtype=torch.float64)
        h0 = zero if st["h0"] is None else st["h0"].double()
        if op == "prompt":
            return _scan64(q, k, v, lam, h0, sc)
        do = st["do"].double()
        dS = zero if st["dhT"] is None else st["dhT"].double()
        dq, _ = _scan64(do, v, k, lam, h0.transpose(2, 3), sc)
        dk, dv = [], []
        for t in range(T - 1, -1, -1):
            dS = dS + sc * (q[:, t, :, :, None] * do[:, t, :, None, :])     # dL/dS_t
            dk.append((dS @ v[:, t, :, :, None])[..., 0])
            dv.append((k[:, t, :, None, :] @ dS)[:, :, 0])
            dS = lam * dS                                                    # dL/dS_{t-1}
        out = []
        for d, n in ((dq, "Hq"), (torch.stack(dk[::-1], 1), "Hk"), (torch.stack(dv[::-1], 1), "Hv")):
            out.append(d.unflatten(2, (case[n], H // case[n])).sum(3))
        return out + ([dS] if st["h0"] is not None else [])
    if op in ("norm", "norm_grad"):
        N, L, C, G = (case[n] for n in ("N", "L", "C", "G"))
        x, w, b = (st[n].double().requires_grad_() for n in ("x", "w", "b"))
        z = None if st["gate"] is None else st["gate"].double().requires_grad_()
        xg = x.view(N, L, G, C // G)
        var, mean = torch.var_mean(xg, (1, 3), unbiased=False)
        rstd = 1 / torch.sqrt(var + st["eps"])
        if op == "norm_grad":     # the stored statistics are inputs of the gradient
            mean = mean + (st["mean"].double() - mean).detach()
            rstd = rstd + (st["rstd"].double() - rstd).detach()
        u = ((xg - mean.view(N, 1, G, 1)) * rstd.view(N, 1, G, 1)).view(N, L, C) * w + b
        f = {"none": lambda t: t, "silu": torch.nn.functional.silu,
             "gelu": torch.nn.functional.gelu}[case["act"]]
        y = f(u) if z is None else u * f(z)
        if op == "norm":
            return y.detach(), mean.detach(), rstd.detach()
        return list(torch.autograd.grad(y, [x, w, b] + ([z] if z is not None else []),
                                        st["dy"].double()))
    # pages: request by request on the host
    P, R, M = case["P"], case["R"], case["M"]
    meta = st["meta"].tolist()
    table = [meta[r * M:(r + 1) * M] for r in range(R)]
    free = meta[R * M:R * M + P]
    n = meta[-1]
    pool = st["pool"]
    if op == "fork":
        for a, c in zip(st["parents"].tolist(), st["children"].tolist()):
            for m in range(M):
                if table[a][m] >= 0:
                    n -= 1
                    table[c][m] = free[n]
                    pool[free[n]] = pool[table[a][m]]
    else:
        used = sorted(p for row in table for p in row if p >= 0)
        holes = sorted(set(range(len(used))) - set(used))
        to = dict(zip([p for p in used if p >= len(used)], holes))
        for a, c in to.items():
            pool[c] = pool[a]
        table = [[to.get(p, p) for p in row] for row in table]
        n = P - len(used)
        free = [P - 1 - i if i < n else -1 for i in range(P)]
    flat = [p for row in table for p in row] + free + [n]
    return pool, torch.tensor(flat, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    es = 2 if case.get("io") == "bf16" else 4
    if op in ("prompt", "grad", "step"):
        H, Hq, Hk, Hv, Dk, Dv = (case[n] for n in ("H", "Hq", "Hk", "Hv", "Dk", "Dv"))
        tokens = case["R"] if op == "step" else case["B"] * case["T"]
        ins = (Hq + Hk) * Dk + Hv * Dv
        if op == "step":
            rows = tokens - (tokens // 16 if tokens > 16 else 0)
            return dict(bytes=rows * (es * (ins + H * Dv) + 8 * H * Dk * Dv),
                        flops=5 * rows * H * Dk * Dv)
        states = case["B"] * H * Dk * Dv * 4
        if op == "prompt":
            return dict(bytes=tokens * es * (ins + H * Dv) + states * (2 if case["state"] else 1),
                        flops=4 * tokens * H * Dk * Dv)
        return dict(bytes=tokens * es * (2 * ins + H * Dv) + states * (3 if case["state"] else 0),
                    flops=10 * tokens * H * Dk * Dv)
    if op in ("norm", "norm_grad"):
        n = case["N"] * case["L"] * case["C"]
        if op == "norm":
            return dict(bytes=n * es * (3 if case["gate"] else 2), flops=10 * n)
        return dict(bytes=n * es * (5 if case["gate"] else 3), flops=25 * n)
    if op == "fork":
        moved = case["n"] * case["M"]
    else:                   # live pages above the live count, for pages anywhere in the pool
        live = (case["R"] + 1) // 2 * case["M"]
        moved = live * (case["P"] - live) // case["P"]
    return dict(bytes=8 * moved * case["page"], flops=0)
