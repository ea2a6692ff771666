"""The layers of examples/selective_layer.py against 64-bit forms of the whole stack.

fp32: a stage's value is a sum of at most a few hundred terms (rows of projections of 64 to 96 inputs, states that
remember up to a hundred tokens) whose roundings of 2^-24 come to 3e-5 of the absolute sum at worst, a tenth of
that in the mean; the norms of queries and keys divide by a head's own root mean square, and a stack of two layers
with its sums passes errors on a few times: the rms is held to 1e-3 (gradients, whose own chains are twice as long:
2e-3).

bf16: a layer rounds six times in a row to bf16 (projection, convolution, projections of the scan, its output, the output
projection, the sum with the input), 0.0017 in the rms each, and as often in the parts that enter products: about 0.008 of
a layer's output, 0.012 of the stack's; the rms is held to 2^-5.
"""
import importlib.util
import os

import pytest
import torch

import hda_ref
import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "selective_layer.py")
    spec = importlib.util.spec_from_file_location("selective_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def conv64(x, w, b):
    xs = torch.nn.functional.pad(x, (0, 0, w.shape[1] - 1, 0))
    return torch.nn.functional.silu(b + sum(w[:, j] * xs[:, j:j + x.shape[1]] for j in range(w.shape[1])))


def selective64(layer, p, h):
    x, z = (h @ p["w_in"].t()).chunk(2, dim=-1)
    u = conv64(x, p["conv_w"], p["conv_b"])
    dt, Bm, Cm = (u @ p["w_x"].t()).split([layer.rank, layer.N, layer.N], dim=-1)
    delta = torch.nn.functional.softplus(dt @ p["w_dt"].t() + p["dt_bias"])
    A, s, ys = -torch.exp(p["A_log"]), 0, []
    for t in range(h.shape[1]):
        s = torch.exp(delta[:, t, :, None] * A) * s + (delta[:, t] * u[:, t])[..., None] * Bm[:, t, None]
        ys.append((s * Cm[:, t, None]).sum(-1))
    y = torch.stack(ys, 1) + p["D"] * u
    return (y * torch.nn.functional.silu(z)) @ p["w_out"].t()


def rotary64(layer, p, h):
    y = conv64(h @ p["w_in"].t(), p["conv_w"], p["conv_b"])
    q, k, v = (t.unflatten(-1, (n, layer.D)) for t, n in zip(y.split([n * layer.D for n in layer.heads], -1), layer.heads))
    T = h.shape[1]
    c, s = (t.double().cpu()[:T][None, :, None] for t in (layer.cos, layer.sin))

    def turned(x, w):
        n = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w
        a, b = n.chunk(2, -1)
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    H = layer.heads[2]
    q, k, v = (hda_ref.wide(t, H) for t in (turned(q, p["wq"]), turned(k, p["wk"]), v))
    lam = torch.exp(layer.decay.double().cpu())[:, None, None]
    S = torch.zeros(h.shape[0], H, layer.D, layer.D, dtype=torch.float64)
    return (layer.scale * hda_ref.scan(q, k, v, lam, S)[0]).flatten(2) @ p["w_out"].t()


def plain(ex, stack, h, params):
    for layer, p in zip(stack.layers, params):
        h = h + (selective64 if isinstance(layer, ex.SelectiveLayer) else rotary64)(layer, p, h)
    return h


def doubles(stack, grad=False):
    return [{n: p.detach().cpu().double().requires_grad_(grad) for n, p in layer.named_parameters()} for layer in stack.layers]


def rms(out, want):
    out = out.detach().cpu().double()
    assert torch.isfinite(out).all()
    return ((out - want).square().mean() / want.square().mean()).sqrt().item()


@pytest.mark.parametrize("C,N,Hq,Hk,D", [(96, 16, 4, 2, 64), (40, 8, 1, 1, 32)])
def test_training_step(ex, C, N, Hq, Hk, D):
    torch.manual_seed(1)
    stack = ex.Stack(ex.SelectiveLayer(64, C, N, dtype=torch.float32),
                     ex.RotaryLayer(64, 4, Hq, Hk, D, dtype=torch.float32))
    x = torch.randn(2, 90, 64, device="cuda", requires_grad=True)
    dy = torch.randn(2, 90, 64, device="cuda")
    y = stack(x)
    y.backward(dy)
    ps = doubles(stack, True)
    x64 = x.detach().cpu().double().requires_grad_(True)
    want = plain(ex, stack, x64, ps)
    want.backward(dy.cpu().double())
    assert rms(y, want.detach()) <= 1e-3
    assert rms(x.grad, x64.grad) <= 2e-3
    for layer, p in zip(stack.layers, ps):
        for n, t in layer.named_parameters():
            assert rms(t.grad, p[n].grad) <= 2e-3, n


@pytest.mark.parametrize("T", [1, 2, 150])
@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 2.0 ** -5)])
def test_serving(ex, T, dtype, tol):
    """Beams of a prompt, stepped and dropped, against the whole sequences."""
    torch.manual_seed(2)
    B, n = 3, 6
    stack = ex.Stack(ex.SelectiveLayer(64, 128, dtype=dtype), ex.RotaryLayer(64, 4, 2, 1, 64, dtype=dtype))
    x = torch.randn(B, T, 64, device="cuda", dtype=dtype)
    tokens = torch.randn(2 * B, n, 64, device="cuda", dtype=dtype)
    out, pages = ex.serve(stack, x, tokens)
    seqs = torch.cat((torch.cat((x, x)), tokens), 1).cpu().double()
    want = plain(ex, stack, seqs, doubles(stack))[:, -n:]
    assert rms(out[B:], want[B:]) <= tol
    assert rms(out[:B, :n // 2], want[:B, :n // 2]) <= tol
    # a dropped row's layers add nothing
    assert torch.equal(out[:B, n // 2:], tokens[:B, n // 2:])
    for p in pages:
        assert p.slots().tolist()[:B] == [-1] * B and p.count.item() == 2 * B


def test_the_example_runs(ex):
    ex.main()


def test_a_decode_step_in_a_graph(ex):
    """All of a step of both layers, captured and replayed, against the same calls one by one."""
    from chunkwise_recurrent_prefill_gb300 import last_device_status
    torch.manual_seed(3)
    stack = ex.Stack(ex.SelectiveLayer(64, 128), ex.RotaryLayer(64, 4, 2, 2, 64))
    x = torch.randn(2, 30, 64, device="cuda", dtype=torch.bfloat16)
    tok = torch.randn(2, 64, device="cuda", dtype=torch.bfloat16)
    pos = torch.full((2,), 30, dtype=torch.int32, device="cuda")

    def fresh():
        pages = [layer.pages(4, 2) for layer in stack.layers]
        stack.prompt(x, pages)
        return pages

    one, two = fresh(), fresh()
    want = [stack.step(tok, one, pos + t) for t in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stack.step(tok, fresh(), pos)           # (libraries of the projections are set up outside of the capture)
    torch.cuda.synchronize()
    at = pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = stack.step(tok, two, at)
    for t in range(3):
        at.copy_(pos + t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[t])
    assert last_device_status() == 0
    for a, b in zip(one, two):
        assert torch.equal(a.states, b.states) and torch.equal(a.tails, b.tails)


def test_two_graphs_at_once():
    """Graphs captured from one stream, with workspaces of the caller's, replayed on two streams."""
    from chunkwise_recurrent_prefill_gb300 import (conv_bwd, conv_workspace_size, qk_norm_bwd, qk_norm_workspace_size,
                                                   ssm_bwd, ssm_workspace_size)
    g = torch.Generator().manual_seed(5)

    def inputs():
        r = lambda *s: ref.gpu(ref.draw(g, *s, io="bf16"))      # noqa: E731
        f = lambda *s: ref.gpu(ref.draw(g, *s))                 # noqa: E731
        d = dict(x=r(2, 500, 64), dy=r(2, 500, 64), w=f(64, 4), dt=r(2, 500, 64), A=-f(64, 16).abs(), B=r(2, 500, 1, 16),
                 C=r(2, 500, 1, 16), q=r(2, 500, 4, 64), k=r(2, 500, 2, 64), wq=f(64), rq=f(2, 500, 4).abs(), rk=f(2, 500, 2).abs())
        sizes = (conv_workspace_size(d["x"], d["w"]), ssm_workspace_size(d["x"], d["dt"], d["A"], d["B"], d["C"], backward=True),
                 qk_norm_workspace_size(d["q"], d["k"]))
        return d, [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]

    def run(d, ws):
        return (*conv_bwd(d["dy"], d["x"], d["w"], act="silu", workspace=ws[0])[:2],
                *ssm_bwd(d["dy"], d["x"], d["dt"], d["A"], d["B"], d["C"], workspace=ws[1])[:5],
                *qk_norm_bwd(d["q"], d["k"], d["q"], d["k"], d["rq"], d["rk"], d["wq"], d["wq"], workspace=ws[2]))

    side, sets, graphs, outs, wants = torch.cuda.Stream(), [inputs(), inputs()], [], [], []
    for d, ws in sets:
        wants.append(run(d, ws))
    torch.cuda.synchronize()
    for d, ws in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(run(d, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for t in (*outs[0], *outs[1]):
            t.zero_()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, wants):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def _chain(x, wait, d):
    """Each call reads what the one before it wrote, into memory that others have just given back."""
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd, hda_fwd, qk_norm_bwd, qk_norm_fwd, ssm_bwd, ssm_fwd
    for _ in range(3):
        y = wait(conv_fwd(x, d["w"], act="silu"))[0]
        o = wait(ssm_fwd(y, d["dt"], d["A"], d["B"], d["C"]))[0]
        q = o.unflatten(-1, (4, 64))
        qo, ko, rq, rk = wait(qk_norm_fwd(q, q[:, :, :2], d["wq"], None, cos=d["cos"], sin=d["sin"]))
        a = wait(hda_fwd(qo, ko, q, d["decay"], 0.1))[0]
        dq, _, dw, _ = wait(qk_norm_bwd(a, ko, q, q[:, :, :2], rq, rk, d["wq"], None, cos=d["cos"], sin=d["sin"]))
        g = wait(ssm_bwd(dq.flatten(2), y, d["dt"], d["A"], d["B"], d["C"]))
        dx, dcw = wait(conv_bwd(g[0], x, d["w"], act="silu"))[:2]
        x = wait((x + dx * 0.1,))[0]
    return x, a, dw, dcw, g[2], g[3]


def _chain_inputs(T=3000):
    g = torch.Generator().manual_seed(7)
    r = lambda *s: ref.gpu(ref.draw(g, *s, io="bf16"))      # noqa: E731
    f = lambda *s: ref.gpu(ref.draw(g, *s))                 # noqa: E731
    ang = torch.arange(T)[:, None] * 0.01 * torch.arange(32)
    return r(2, T, 256), dict(w=f(256, 4), dt=r(2, T, 256).abs() * 0.1, A=-f(256, 16).abs(), B=r(2, T, 1, 16), C=r(2, T, 1, 16),
                              wq=f(64), cos=ref.gpu(torch.cos(ang)), sin=ref.gpu(torch.sin(ang)), decay=-f(4).abs() * 0.1)


def test_calls_behind_each_other():
    """Kernels are scheduled before those ahead of them in the stream are done: nothing may be read or written early."""
    x, d = _chain_inputs()

    def sync(r):
        torch.cuda.synchronize()
        return r

    want = _chain(x, sync, d)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(_chain(x, lambda r: r, d), want))


def test_a_capture_of_two_streams():
    """A capture that forks and joins: the kernel behind the join waits for both."""
    from chunkwise_recurrent_prefill_gb300 import conv_fwd, qk_norm_fwd, ssm_fwd
    x, d = _chain_inputs(1000)

    def run(main, other):
        y, _ = conv_fwd(x, d["w"], act="silu")
        other.wait_stream(main)
        with torch.cuda.stream(other):
            dt = conv_fwd(d["dt"], d["w"].abs() * 0.1)[0].abs()
            q = qk_norm_fwd(x.unflatten(-1, (4, 64)), y.unflatten(-1, (4, 64)))[1].flatten(2)
        z = conv_fwd(y, d["w"])[0]
        main.wait_stream(other)
        return ssm_fwd(q, dt, d["A"], d["B"], d["C"], z=z)[0]

    other = torch.cuda.Stream()
    want = run(torch.cuda.current_stream(), other)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run(side, other)                # (its workspace; a call that is captured makes none)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = run(side, other)
    for _ in range(10):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_calls_of_two_threads():
    """Calls of one kernel that need different amounts of shared memory, from threads with a stream each."""
    import threading
    from chunkwise_recurrent_prefill_gb300 import qk_norm_bwd, qk_norm_fwd, ssm_bwd, ssm_fwd
    g = torch.Generator().manual_seed(9)
    f = lambda *s: ref.gpu(ref.draw(g, *s))                 # noqa: E731

    def inputs(T, N, D):
        return dict(u=f(1, T, 64), dt=f(1, T, 64), A=-f(64, N).abs(), B=f(1, T, 1, N), C=f(1, T, 1, N), q=f(1, T, 2, D), w=f(D))

    def run(d):
        o = ssm_fwd(d["u"], d["dt"], d["A"], d["B"], d["C"])[0]
        du = ssm_bwd(o, d["u"], d["dt"], d["A"], d["B"], d["C"])[:5]
        qo, ko, rq, rk = qk_norm_fwd(d["q"], d["q"], d["w"], d["w"])
        return (o, *du, qo, *qk_norm_bwd(qo, ko, d["q"], d["q"], rq, rk, d["w"], d["w"]))

    sets = [inputs(9, 20, 24), inputs(300, 128, 300), inputs(40, 40, 999)]
    wants = [run(d) for d in sets]
    torch.cuda.synchronize()
    failed = []

    def work(d, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(100):
                    got = run(d)
                torch.cuda.current_stream().synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want))
        except Exception as e:      # noqa: BLE001 (reported by the test's own thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(sets, wants)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
