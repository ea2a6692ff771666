"""Plain 64-bit forms of the decay attention, token by token, and the bounds its kernels are
held to.

Every output is a sum of products of inputs, decayed along the way. With u = 2^-24 and A the
same sum over absolute values, K successive fp32 roundings of each term leave an error of at
most K u A (to first order):

* token by token: a term is multiplied by the decay once per later token (the product, the
  addition of the new term, and the decay's own two roundings: 4 per token) and added across
  Dx / 8 rows and three shuffles: K = 4 T + Dx / 8 + 16.
* tensor cores: the same fp32 work, and roundings to bf16 (2^-8 of a term at most): one of the
  masked score or of the state's snapshot for an output. The state's update carries its operand
  in two bf16 parts or more, which leaves 2^-16 of a term at most.

bf16 outputs add their own rounding, 2^-8 of the value. The roundings of a bf16 output are
independent, so their joint effect over a tensor is much smaller than A says: each has a
relative deviation of about 2^-8 / sqrt(12) * 1.5 = 0.0017, and three of them 0.0029, so the
root mean square of the error is also held to 2^-8 = 0.0039 of that of the output.
"""
import torch

U = 2.0 ** -24


def wide(t, H):
    """[B, T, heads, D] -> float64 [B, T, H, D]."""
    return t.double().repeat_interleave(H // t.shape[2], 2)


def scan(x, y, z, lam, S):
    out = []
    for t in range(x.shape[1]):
        S = lam * S + y[:, t, :, :, None] * z[:, t, :, None, :]
        out.append(torch.einsum("bhx,bhxz->bhz", x[:, t], S))
    return (torch.stack(out, 1) if out else x.new_zeros(x.shape[:3] + z.shape[3:])), S


def forward(q, k, v, decay, scale, h0=None):
    """o [B,T,H,Dv], hT in float64 of CPU tensors."""
    H = decay.numel()
    q, k, v = wide(q, H), wide(k, H), wide(v, H)
    lam = torch.exp(decay.double())[:, None, None]
    S = torch.zeros(q.shape[0], H, q.shape[3], v.shape[3], dtype=torch.float64) if h0 is None else h0.double()
    o, S = scan(q, k, v, lam, S)
    return scale * o, S


def backward(do, q, k, v, decay, scale, h0=None, dhT=None):
    """dq, dk, dv (summed over shared heads) and dh0, by the formulas, in float64."""
    H = decay.numel()
    nq, nk, nv = q.shape[2], k.shape[2], v.shape[2]
    q, k, v, do = wide(q, H), wide(k, H), wide(v, H), do.double()
    lam = torch.exp(decay.double())[:, None, None]
    zero = torch.zeros(q.shape[0], H, q.shape[3], v.shape[3], dtype=torch.float64)
    S = zero if h0 is None else h0.double()
    dS = zero if dhT is None else dhT.double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(q.shape[1]):
        S = lam * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        dq[:, t] = scale * torch.einsum("bhxz,bhz->bhx", S, do[:, t])
    for t in range(q.shape[1] - 1, -1, -1):
        dS = dS + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dk[:, t] = torch.einsum("bhxz,bhz->bhx", dS, v[:, t])
        dv[:, t] = torch.einsum("bhxz,bhx->bhz", dS, k[:, t])
        dS = lam * dS
    share = lambda d, n: d.unflatten(2, (n, H // n)).sum(3)  # noqa: E731
    return share(dq, nq), share(dk, nk), share(dv, nv), dS


def roundings(T, D):
    return 4 * T + D / 8 + 16


def check(name, out, ref, absolute, T, D, path="exact", state=False):
    """out against ref within the bounds above; absolute: the same map of absolute values."""
    out64, bf16 = out.detach().cpu().double(), out.dtype == torch.bfloat16
    per_term = roundings(T, D) * U
    if path == "tc":
        per_term += 2.0 ** -16 if state else 2.0 ** -8
    bound = per_term * absolute + (2.0 ** -8 * ref.abs() if bf16 else 0.0) + 1e-37
    err = (out64 - ref).abs()
    assert torch.isfinite(out64).all(), f"{name}: not finite"
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"
    if bf16 and ref.numel() >= 4096:
        rms = (err.square().mean() / ref.square().mean()).sqrt().item()
        assert rms <= 2.0 ** -8, f"{name}: rms error {rms:.3g} of the output's"


def inputs(B, T, H, Hq, Hk, Hv, Dk, Dv, io="bf16", seed=0, decay=None, strided=False):
    """CPU tensors q, k, v, do, decay, h0, dhT; strided: q, k, v are slices of one tensor."""
    g = torch.Generator("cpu").manual_seed(seed)
    dt = torch.bfloat16 if io == "bf16" else torch.float32
    qkv = torch.randn(B, T, Hq * Dk + Hk * Dk + Hv * Dv, generator=g).to(dt)
    q, k, v = qkv.split([Hq * Dk, Hk * Dk, Hv * Dv], dim=-1)
    q, k, v = q.unflatten(-1, (Hq, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (Hv, Dv))
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    do = torch.randn(B, T, H, Dv, generator=g).to(dt)
    if decay is None:
        decay = [-2.0 ** (-8.0 * (h + 1) / max(H, 2)) for h in range(H)]
    return dict(q=q, k=k, v=v, do=do, decay=torch.tensor(decay, dtype=torch.float32),
                h0=torch.randn(B, H, Dk, Dv, generator=g), dhT=torch.randn(B, H, Dk, Dv, generator=g),
                scale=Dk ** -0.5)


def to_gpu(t):
    """A CUDA copy that keeps the strides (of slices of one tensor, too)."""
    if t is None or not isinstance(t, torch.Tensor) or t.is_contiguous():
        return t.cuda() if isinstance(t, torch.Tensor) else t
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    base.copy_(t)
    return base
