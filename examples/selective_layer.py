"""Two recurrent layers with a short convolution in front, as they are trained and served.

    SelectiveLayer   x, z = h W_in;  x = silu(conv(x));  dt, B, C = x W_x;  y = scan(x, dt, B, C) silu(z);  y W_out
    RotaryLayer      q, k, v = silu(conv(h W_in));  q, k = rotated norms per head;  o = decay attention;  o W_out

Training runs the pairs ``conv_fwd`` / ``conv_bwd``, ``ssm_fwd`` / ``ssm_bwd``, ``qk_norm_fwd`` / ``qk_norm_bwd`` and
``hda_fwd`` / ``hda_bwd``. Serving keeps a row's last inputs and its state in the same page of two pools: the prompt writes
them, ``conv_step`` and ``ssm_step`` (``hda_step``) advance them in place, ``pages_fork`` makes beams of them.

    python examples/selective_layer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from chunkwise_recurrent_prefill_gb300 import (  # noqa: E402
    conv_bwd, conv_fwd, conv_step, hda_bwd, hda_fwd, hda_step, last_device_status, pages_copy, pages_fork, pages_free,
    qk_norm_bwd, qk_norm_fwd, ssm_bwd, ssm_fwd, ssm_step)


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias):
        ctx.save_for_backward(x, w, bias)
        return conv_fwd(x, w, bias, act="silu")[0]

    @staticmethod
    def backward(ctx, dy):
        return conv_bwd(dy.contiguous(), *ctx.saved_tensors, act="silu")[:3]


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, Bm, Cm, D, z, dt_bias):
        ctx.save_for_backward(u, dt, A, Bm, Cm, D, z, dt_bias)
        return ssm_fwd(u, dt, A, Bm, Cm, D=D, z=z, dt_bias=dt_bias)[0]

    @staticmethod
    def backward(ctx, do):
        u, dt, A, Bm, Cm, D, z, dt_bias = ctx.saved_tensors
        return ssm_bwd(do.contiguous(), u, dt, A, Bm, Cm, D=D, z=z, dt_bias=dt_bias)[:8]


class RotatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cos, sin):
        qo, ko, rq, rk = qk_norm_fwd(q, k, wq, wk, cos=cos, sin=sin)
        ctx.save_for_backward(q, k, rq, rk, wq, wk, cos, sin)
        return qo, ko

    @staticmethod
    def backward(ctx, dqo, dko):
        q, k, rq, rk, wq, wk, cos, sin = ctx.saved_tensors
        return (*qk_norm_bwd(dqo.contiguous(), dko.contiguous(), q, k, rq, rk, wq, wk, cos=cos, sin=sin), None, None)


class DecayAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, decay, scale):
        ctx.save_for_backward(q, k, v, decay)
        ctx.scale = scale
        return hda_fwd(q, k, v, decay, scale)[0]

    @staticmethod
    def backward(ctx, do):
        return (*hda_bwd(do.contiguous(), *ctx.saved_tensors, ctx.scale)[:3], None, None)


def _matrix(out, inner, dtype, device):
    return torch.nn.Parameter((torch.randn(out, inner, device=device) * inner ** -0.5).to(dtype))


class Pages:
    """P pages of one layer: the last inputs of its convolution and its states. Row r of R has page table[r] (-1: none)."""

    def __init__(self, P, R, tail, state, dtype, device="cuda"):
        self.tails = torch.zeros(P, *tail, dtype=dtype, device=device)
        self.states = torch.zeros(P, *state, device=device)
        self.table = torch.full((R, 1), -1, dtype=torch.int32, device=device)
        self.free = torch.arange(P - 1, -1, -1, dtype=torch.int32, device=device)
        self.count = torch.full((1,), P, dtype=torch.int32, device=device)

    def admit(self, B):
        """Rows 0 .. B-1 of unused pages take the first B."""
        self.table[:B, 0] = torch.arange(B, dtype=torch.int32, device=self.table.device)
        self.count -= B
        return self.tails[:B], self.states[:B]

    def slots(self):
        return self.table.view(-1)

    def fork(self, parents, children):
        pages_fork(self.states, self.table, self.free, self.count, parents, children)
        pages_copy(self.tails, self.table[parents.long(), 0], self.table[children.long(), 0])

    def drop(self, rows):
        pages_free(self.table, self.free, self.count, rows)


class SelectiveLayer(torch.nn.Module):
    """C channels of N states; step sizes from a projection of rank ``rank``."""

    def __init__(self, width, C, N=16, rank=None, W=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.C, self.N, self.W, self.rank, self.dtype = C, N, W, rank or max(1, C // 16), dtype
        self.w_in, self.w_x = _matrix(2 * C, width, dtype, device), _matrix(self.rank + 2 * N, C, dtype, device)
        self.w_dt, self.w_out = _matrix(C, self.rank, dtype, device), _matrix(width, C, dtype, device)
        self.conv_w = torch.nn.Parameter(torch.randn(C, W, device=device) * W ** -0.5)
        self.conv_b = torch.nn.Parameter(torch.zeros(C, device=device))
        self.A_log = torch.nn.Parameter(torch.log(torch.arange(1, N + 1, device=device).float()).repeat(C, 1))
        self.D = torch.nn.Parameter(torch.ones(C, device=device))
        step = torch.exp(torch.rand(C, device=device) * math.log(100.0) + math.log(1e-3))   # 0.001 to 0.1
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))

    def pages(self, P, R):
        return Pages(P, R, (self.W - 1, self.C), (self.C, self.N), self.dtype, self.D.device)

    def inputs(self, u):
        """dt, B and C of u, views of one projection."""
        dt, Bm, Cm = (u @ self.w_x.t()).split([self.rank, self.N, self.N], dim=-1)
        return dt @ self.w_dt.t(), Bm.unsqueeze(-2), Cm.unsqueeze(-2)

    def forward(self, h):
        x, z = (h @ self.w_in.t()).chunk(2, dim=-1)
        u = Conv.apply(x, self.conv_w, self.conv_b)
        dt, Bm, Cm = self.inputs(u)
        return Scan.apply(u, dt, -torch.exp(self.A_log), Bm, Cm, self.D, z, self.dt_bias) @ self.w_out.t()

    @torch.no_grad()
    def prompt(self, h, pages):
        tails, states = pages.admit(h.shape[0])
        x, z = (h @ self.w_in.t()).chunk(2, dim=-1)
        u, _ = conv_fwd(x, self.conv_w, self.conv_b, act="silu", sT=tails)
        dt, Bm, Cm = self.inputs(u)
        o, _ = ssm_fwd(u, dt, -torch.exp(self.A_log), Bm, Cm, D=self.D, z=z, dt_bias=self.dt_bias, hT=states)
        return o @ self.w_out.t()

    @torch.no_grad()
    def step(self, h, pages, positions):
        x, z = (h @ self.w_in.t()).chunk(2, dim=-1)
        u = conv_step(x, self.conv_w, pages.tails, pages.slots(), self.conv_b, act="silu")
        dt, Bm, Cm = self.inputs(u)
        o = ssm_step(u, dt, -torch.exp(self.A_log), Bm, Cm, pages.states, pages.slots(), D=self.D, z=z,
                     dt_bias=self.dt_bias)
        return o @ self.w_out.t()


class RotaryLayer(torch.nn.Module):
    """H states of D x D with a decay each; queries and keys have Hq and Hk heads (divisors of H)."""

    def __init__(self, width, H, Hq, Hk, D, W=4, most=4096, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.D, self.W, self.dtype, self.scale = (Hq, Hk, H), D, W, dtype, D ** -0.5
        rows = (Hq + Hk + H) * D
        self.w_in, self.w_out = _matrix(rows, width, dtype, device), _matrix(width, H * D, dtype, device)
        self.conv_w = torch.nn.Parameter(torch.randn(rows, W, device=device) * W ** -0.5)
        self.conv_b = torch.nn.Parameter(torch.zeros(rows, device=device))
        self.wq = torch.nn.Parameter(torch.ones(D, device=device))
        self.wk = torch.nn.Parameter(torch.ones(D, device=device))
        self.register_buffer("decay", -torch.exp2(-torch.linspace(2.5, 8.0, H, device=device)))
        angle = torch.arange(most, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(D // 2) * 2.0 / D)
        self.register_buffer("cos", torch.cos(angle).float().to(device))
        self.register_buffer("sin", torch.sin(angle).float().to(device))

    def pages(self, P, R):
        H, D = self.heads[2], self.D
        return Pages(P, R, (self.W - 1, self.conv_w.shape[0]), (H, D, D), self.dtype, self.decay.device)

    def split(self, y):
        return (t.unflatten(-1, (n, self.D)) for t, n in
                zip(y.split([n * self.D for n in self.heads], dim=-1), self.heads))

    def forward(self, h):
        q, k, v = self.split(Conv.apply(h @ self.w_in.t(), self.conv_w, self.conv_b))
        q, k = RotatedNorm.apply(q, k, self.wq, self.wk, self.cos, self.sin)
        return DecayAttention.apply(q, k, v, self.decay, self.scale).flatten(-2) @ self.w_out.t()

    @torch.no_grad()
    def prompt(self, h, pages):
        tails, states = pages.admit(h.shape[0])
        q, k, v = self.split(conv_fwd(h @ self.w_in.t(), self.conv_w, self.conv_b, act="silu", sT=tails)[0])
        q, k, _, _ = qk_norm_fwd(q, k, self.wq, self.wk, cos=self.cos, sin=self.sin)
        return hda_fwd(q, k, v, self.decay, self.scale, hT=states)[0].flatten(-2) @ self.w_out.t()

    @torch.no_grad()
    def step(self, h, pages, positions):
        y = conv_step(h @ self.w_in.t(), self.conv_w, pages.tails, pages.slots(), self.conv_b, act="silu")
        q, k, v = self.split(y)
        q, k, _, _ = qk_norm_fwd(q[:, None], k[:, None], self.wq, self.wk, cos=self.cos, sin=self.sin,
                                 positions=positions[:, None])
        o = hda_step(q[:, 0], k[:, 0], v, self.decay, self.scale, pages.states, pages.slots())
        return o.flatten(-2) @ self.w_out.t()


class Stack(torch.nn.Module):
    """Layers one behind the other, each added to its input."""

    def __init__(self, *layers):
        super().__init__()
        self.layers = torch.nn.ModuleList(layers)

    def forward(self, h):
        for layer in self.layers:
            h = h + layer(h)
        return h

    def prompt(self, h, pages):
        for layer, p in zip(self.layers, pages):
            h = h + layer.prompt(h, p)
        return h

    def step(self, h, pages, positions):
        for layer, p in zip(self.layers, pages):
            h = h + layer.step(h, p, positions)
        return h


def train(stack, x, target, steps=3, lr=1e-3):
    """A few steps of plain gradient descent; the losses."""
    losses = []
    for _ in range(steps):
        loss = (stack(x).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in stack.parameters():
                p.sub_(p.grad, alpha=lr)
                p.grad = None
        losses.append(loss.item())
    return losses


def serve(stack, prompt, tokens):
    """A prompt [B, T, width], two beams of each row, the steps tokens [2 B, n, width]; after half of them the
    first beam of every row is dropped. Returns the steps' outputs [2 B, n, width] and the pages."""
    (B, T), n, dev = prompt.shape[:2], tokens.shape[1], prompt.device
    pages = [layer.pages(3 * B, 2 * B) for layer in stack.layers]
    stack.prompt(prompt, pages)
    first = torch.arange(B, dtype=torch.int32, device=dev)
    for p in pages:
        p.fork(first, first + B)
    out = []
    for t in range(n):
        if t == n // 2:
            for p in pages:
                p.drop(first)
        positions = torch.full((2 * B,), T + t, dtype=torch.int32, device=dev)
        out.append(stack.step(tokens[:, t], pages, positions))
    return torch.stack(out, 1), pages


def main():
    torch.manual_seed(0)
    stack = Stack(SelectiveLayer(512, 1024), RotaryLayer(512, H=8, Hq=8, Hk=2, D=64))
    x = torch.randn(2, 200, 512, device="cuda", dtype=torch.bfloat16)
    losses = train(stack, x, torch.randn(2, 200, 512, device="cuda"))
    print("losses", " ".join(f"{v:.5f}" for v in losses))
    tokens = torch.randn(4, 6, 512, device="cuda", dtype=torch.bfloat16)
    out, pages = serve(stack, x, tokens)
    with torch.no_grad():       # the second beams have seen the prompt and all six tokens
        whole = stack(torch.cat((x, tokens[2:]), 1))[:, -6:].float()
    err = ((out[2:].float() - whole).square().mean() / whole.square().mean()).sqrt().item()
    print(f"steps against the whole sequence: rms difference {err:.5f}")
    print("pages of the rows", [p.slots().tolist() for p in pages])
    assert last_device_status() == 0
    assert err < 2.0 ** -5


if __name__ == "__main__":
    main()
