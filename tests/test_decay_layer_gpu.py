"""The layer of examples/decay_layer.py against a 64-bit form of the whole layer.

fp32: each value of a stage is a sum of at most T = 130 decayed terms or a row of a projection,
and carries a few hundred roundings of 2^-24 of its absolute sum at worst, 3e-5, about a tenth of
that in the mean. The norm divides by a head's own root mean square, so the few of the first
tokens whose q k nearly cancels magnify this about a hundredfold: the rms is held to 1e-3.

bf16: each of the projection, the attention, the norm and the output projection rounds once
(0.0017 in the rms) or, the attention, up to 2^-8; with the roundings of q, k and v about 0.006
together, and as much again for the first tokens that cancel: the rms is held to 2^-6.
"""
import importlib.util
import os

import pytest
import torch

import hda_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "decay_layer.py")
    spec = importlib.util.spec_from_file_location("decay_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain(layer, x, w_in, w_out, norm):
    """The layer in float64 on the CPU, differentiable."""
    H, (Hq, Hk, Hv) = layer.H, layer.heads
    q, k, v, z = (x @ w_in.t()).split(layer.sizes, dim=-1)
    q, k, v = (hda_ref.wide(t.unflatten(-1, (n, -1)), H) for t, n in ((q, Hq), (k, Hk), (v, Hv)))
    lam = torch.exp(layer.decay.double().cpu())[:, None, None]
    S = torch.zeros(x.shape[0], H, layer.Dk, layer.Dv, dtype=torch.float64)
    o = layer.scale * hda_ref.scan(q, k, v, lam, S)[0]
    mean = o.mean(-1, keepdim=True)
    xhat = (o - mean) / ((o - mean).square().mean(-1, keepdim=True) + 1e-5).sqrt()
    return (xhat.flatten(2) * norm * torch.nn.functional.silu(z)) @ w_out.t()


def doubles(layer, grad=False):
    return [p.detach().cpu().double().requires_grad_(grad) for p in (layer.w_in, layer.w_out, layer.norm)]


def rms(out, ref):
    out = out.detach().cpu().double()
    assert torch.isfinite(out).all()
    return ((out - ref).square().mean() / ref.square().mean()).sqrt().item()


@pytest.mark.parametrize("Hq,Hk,Dk,Dv", [(4, 4, 64, 64), (2, 1, 64, 128)])
def test_training_step(ex, Hq, Hk, Dk, Dv):
    torch.manual_seed(1)
    layer = ex.DecayLayer(96, 4, Hq, Hk, Dk, Dv, dtype=torch.float32)
    x = torch.randn(2, 130, 96, device="cuda", requires_grad=True)
    dy = torch.randn(2, 130, 96, device="cuda")
    y = layer(x)
    y.backward(dy)
    ps = doubles(layer, True)
    x64 = x.detach().cpu().double().requires_grad_(True)
    ref = plain(layer, x64, *ps)
    ref.backward(dy.cpu().double())
    assert rms(y, ref.detach()) <= 1e-3
    for name, g, r in (("x", x, x64), ("w_in", layer.w_in, ps[0]), ("w_out", layer.w_out, ps[1]),
                       ("norm", layer.norm, ps[2])):
        assert rms(g.grad, r.grad) <= 1e-3, name


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 2.0 ** -6)])
def test_serving(ex, T, dtype, tol):
    """Beams of a prompt, stepped, dropped and compacted, against the whole sequences."""
    torch.manual_seed(2)
    B, n = 3, 6
    layer = ex.DecayLayer(128, 8, 4, 2, 128, 128, dtype=dtype)
    x = torch.randn(B, T, 128, device="cuda", dtype=dtype)
    tokens = torch.randn(2 * B, n, 128, device="cuda", dtype=dtype)
    out, pool = ex.serve(layer, x, tokens)
    seqs = torch.cat((torch.cat((x, x)), tokens), 1).cpu().double()
    ref = plain(layer, seqs, *doubles(layer))[:, -n:]
    assert rms(out[B:], ref[B:]) <= tol
    assert rms(out[:B, :n // 2], ref[:B, :n // 2]) <= tol
    assert not out[:B, n // 2:].any()
    slots = pool.slots().tolist()
    assert slots[:B] == [-1] * B and sorted(slots[B:]) == list(range(B))
    assert pool.count.item() == 2 * B


def test_training_lowers_the_loss(ex):
    torch.manual_seed(3)
    layer = ex.DecayLayer(256, 8, 8, 2, 128, 128)
    x = torch.randn(2, 300, 256, device="cuda", dtype=torch.bfloat16)
    losses = ex.train(layer, x, torch.randn(2, 300, 256, device="cuda"))
    assert losses[-1] < losses[0]


def test_steps_in_a_graph(ex):
    """One decode step's own kernels (fork, step, norm, free, compact), captured and replayed,
    against the same calls one by one."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_fwd, hda_step, last_device_status
    torch.manual_seed(4)
    layer = ex.DecayLayer(64, 4, 2, 2, 64, 64)
    R = 4
    q, k, v, z = layer.split(torch.randn(R, 64, device="cuda", dtype=torch.bfloat16))
    q, k, v, z = (t.detach() for t in (q, k, v, z))
    norm = layer.norm.detach()
    rows = torch.arange(2, dtype=torch.int32, device="cuda")

    def fresh():
        pool = ex.StatePool(layer, 6, R)
        pool.admit(2).copy_(states)
        return pool

    def step(pool):
        pool.fork(rows, rows + 2)
        o = hda_step(q, k, v, layer.decay, layer.scale, pool.pages, pool.slots())
        y, _, _ = group_norm_fwd(o.view(R, -1), layer.H, norm, act="silu", gate=z)
        pool.drop(rows)
        pool.compact()
        return y

    states = torch.randn(2, 4, 64, 64, device="cuda")
    plain = fresh()
    want = step(plain)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):       # the stream's workspace exists before the capture
        step(fresh())
    torch.cuda.current_stream().wait_stream(side)
    pool = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(pool)
    graph.replay()
    torch.cuda.synchronize()
    assert last_device_status() == 0
    assert torch.equal(got, want) and torch.equal(pool.table, plain.table)
    assert torch.equal(pool.pages[:2], plain.pages[:2]) and torch.equal(pool.count, plain.count)
