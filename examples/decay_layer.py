"""One layer of linear attention with a decay per head, as it is trained and served.

    q, k, v, z = x W_in;   o = decay attention(q, k, v);   y = (group norm of o per head) silu(z) W_out

Training runs ``hda_fwd`` / ``hda_bwd`` and ``group_norm_fwd`` / ``group_norm_bwd``. Serving keeps
the state of each row in a page of a pool: ``hda_fwd`` writes a prompt's state into its page,
``pages_fork`` makes beams of it, ``hda_step`` advances every row in place, ``pages_free`` and
``pages_compact`` take the dropped beams out.

    python examples/decay_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from chunkwise_recurrent_prefill_gb300 import (  # noqa: E402
    group_norm_bwd, group_norm_fwd, hda_bwd, hda_fwd, hda_step, last_device_status,
    pages_compact, pages_fork, pages_free)


class DecayAttention(torch.autograd.Function):
    """The decays are constants of the layer and have no gradient."""

    @staticmethod
    def forward(ctx, q, k, v, decay, scale):
        ctx.save_for_backward(q, k, v, decay)
        ctx.scale = scale
        return hda_fwd(q, k, v, decay, scale)[0]

    @staticmethod
    def backward(ctx, do):
        dq, dk, dv, _ = hda_bwd(do.contiguous(), *ctx.saved_tensors, ctx.scale)
        return dq, dk, dv, None, None


class GatedNorm(torch.autograd.Function):
    """silu(z) times the group norm of x [N, C]; z may be a slice of wider rows."""

    @staticmethod
    def forward(ctx, x, z, weight, groups):
        y, mean, rstd = group_norm_fwd(x, groups, weight, act="silu", gate=z)
        ctx.save_for_backward(x, z, weight, mean, rstd)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, z, weight, mean, rstd = ctx.saved_tensors
        dx, dw, _, dz = group_norm_bwd(dy.contiguous(), x, mean, rstd, ctx.groups, weight, act="silu", gate=z)
        return dx, dz, dw, None


class DecayLayer(torch.nn.Module):
    """H states of Dk x Dv; queries and keys may have fewer heads than the states (Hq, Hk
    divide H)."""

    def __init__(self, width, H, Hq, Hk, Dk, Dv, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.H, self.Dk, self.Dv, self.heads = H, Dk, Dv, (Hq, Hk, H)
        self.sizes = (Hq * Dk, Hk * Dk, H * Dv, H * Dv)
        self.w_in = torch.nn.Parameter(
            (torch.randn(sum(self.sizes), width, device=device) * width ** -0.5).to(dtype))
        self.w_out = torch.nn.Parameter(
            (torch.randn(width, H * Dv, device=device) * (H * Dv) ** -0.5).to(dtype))
        self.norm = torch.nn.Parameter(torch.ones(H * Dv, device=device))
        # half-lives from about four tokens to thousands
        self.register_buffer("decay", -torch.exp2(-torch.linspace(2.5, 10.0, H, device=device)))
        self.scale = Dk ** -0.5

    def split(self, x):
        """q [..., Hq, Dk], k, v and the gate z [..., H Dv], all views of one projection."""
        q, k, v, z = (x @ self.w_in.t()).split(self.sizes, dim=-1)
        Hq, Hk, Hv = self.heads
        return q.unflatten(-1, (Hq, self.Dk)), k.unflatten(-1, (Hk, self.Dk)), v.unflatten(-1, (Hv, self.Dv)), z

    def finish(self, o, z):
        """The norm over each head of a token, the gate and the output projection."""
        rows = GatedNorm.apply(o.reshape(-1, self.H * self.Dv), z.reshape(-1, self.H * self.Dv), self.norm, self.H)
        return rows.view(*o.shape[:-2], -1) @ self.w_out.t()

    def forward(self, x):
        """x [B, T, width]."""
        q, k, v, z = self.split(x)
        return self.finish(DecayAttention.apply(q, k, v, self.decay, self.scale), z)

    @torch.no_grad()
    def prompt(self, x, states):
        """As forward; the final states of the B rows go to ``states`` [B, H, Dk, Dv]."""
        q, k, v, z = self.split(x)
        return self.finish(hda_fwd(q, k, v, self.decay, self.scale, hT=states)[0], z)

    @torch.no_grad()
    def step(self, x, pool, slots):
        """One token x [R, width] for each row; row r's state is page slots[r] of the pool."""
        q, k, v, z = self.split(x)
        return self.finish(hda_step(q, k, v, self.decay, self.scale, pool, slots), z)


class StatePool:
    """P pages of one layer's state, one page for each of R rows (-1: none)."""

    def __init__(self, layer, P, R):
        dev = layer.decay.device
        self.pages = torch.zeros(P, layer.H, layer.Dk, layer.Dv, device=dev)
        self.table = torch.full((R, 1), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(P - 1, -1, -1, dtype=torch.int32, device=dev)
        self.count = torch.full((1,), P, dtype=torch.int32, device=dev)

    def admit(self, B):
        """Rows 0 .. B-1 of an unused pool take its first B pages, returned for the prompt's
        states."""
        self.table[:B, 0] = torch.arange(B, dtype=torch.int32, device=self.table.device)
        self.count -= B
        return self.pages[:B]

    def slots(self):
        return self.table.view(-1)

    def fork(self, parents, children):
        pages_fork(self.pages, self.table, self.free, self.count, parents, children)

    def drop(self, rows):
        pages_free(self.table, self.free, self.count, rows)

    def compact(self):
        pages_compact(self.pages, self.table, self.free, self.count)


def train(layer, x, target, steps=3, lr=0.5):
    """A few steps of plain gradient descent; the losses."""
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in layer.parameters():
                p.sub_(p.grad, alpha=lr)
                p.grad = None
        losses.append(loss.item())
    return losses


def serve(layer, prompt, tokens):
    """A prompt [B, T, width], two beams of each row, the steps tokens [2 B, n, width]; after
    half of them the first beam of every row is dropped (its outputs are then zero). Returns the
    outputs of the steps [2 B, n, width] and the pool."""
    B, n = prompt.shape[0], tokens.shape[1]
    dev = prompt.device
    pool = StatePool(layer, 3 * B, 2 * B)
    layer.prompt(prompt, pool.admit(B))
    first = torch.arange(B, dtype=torch.int32, device=dev)
    pool.fork(first, first + B)
    out = []
    for t in range(n):
        if t == n // 2:
            pool.drop(first)
            pool.compact()
        out.append(layer.step(tokens[:, t], pool.pages, pool.slots()))
    return torch.stack(out, 1), pool


def main():
    torch.manual_seed(0)
    layer = DecayLayer(width=512, H=8, Hq=8, Hk=2, Dk=128, Dv=128)
    x = torch.randn(2, 200, 512, device="cuda", dtype=torch.bfloat16)
    losses = train(layer, x, torch.randn(2, 200, 512, device="cuda"))
    print("losses", " ".join(f"{v:.5f}" for v in losses))

    tokens = torch.randn(4, 6, 512, device="cuda", dtype=torch.bfloat16)
    out, pool = serve(layer, x, tokens)
    # the second beams have seen the prompt and all six tokens
    with torch.no_grad():
        whole = layer(torch.cat((x, tokens[2:]), 1))[:, -6:].float()
    err = ((out[2:].float() - whole).square().mean() / whole.square().mean()).sqrt().item()
    print(f"steps against the whole sequence: rms difference {err:.5f}")
    print("pages of the rows", pool.slots().tolist(), "free", pool.count.item())
    assert last_device_status() == 0
    assert losses[-1] < losses[0] and err < 2.0 ** -6
    assert not out[:2, 3:].any() and pool.count.item() == 4


if __name__ == "__main__":
    main()
