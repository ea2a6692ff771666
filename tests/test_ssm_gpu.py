"""Selective state space scan against its 64-bit form (bounds: layer_ref.py)."""
import math

import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu
GRADS = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "dbias", "dh0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def make(B, T, C, G=1, N=16, io="f32", seed=0, z=True, state=True, params=True, strided=False, steps=(1e-3, 0.1)):
    g = torch.Generator().manual_seed(seed)

    def rows(*tail):
        w = math.prod(tail)
        if not strided:
            return ref.draw(g, B, T, *tail, io=io)
        return ref.draw(g, B, T, 2 * w + 3, io=io)[..., 3:3 + w].unflatten(-1, tail)

    step = torch.exp(torch.rand(C, generator=g) * math.log(steps[1] / steps[0]) + math.log(steps[0]))
    return dict(u=rows(C), dt=rows(C), z=rows(C) if z else None, Bm=rows(G, N), Cm=rows(G, N), do=rows(C),
                A=-torch.arange(1, N + 1).float() * torch.exp(0.1 * torch.randn(C, N, generator=g)),
                D=ref.draw(g, C) if params else None,
                dt_bias=step + torch.log(-torch.expm1(-step)) if params else None,
                h0=ref.draw(g, B, C, N) if state else None, dhT=ref.draw(g, B, C, N) if state else None)


def call(t, softplus=True, **kw):
    from chunkwise_recurrent_prefill_gb300 import ssm_bwd, ssm_fwd
    a = (t["u"], t["dt"], t["A"], t["Bm"], t["Cm"])
    k = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"], softplus=softplus, **kw)
    o, hT = ssm_fwd(*a, return_state=True, **k)
    return dict(zip(("o", "hT") + GRADS, (o, hT) + ssm_bwd(t["do"], *a, dhT=t["dhT"], **k)))


def check(d, io, softplus=True, **kw):
    from chunkwise_recurrent_prefill_gb300 import last_device_status
    got = call({n: ref.gpu(v) for n, v in d.items()}, softplus, **kw)
    assert last_device_status() == 0
    want = ref.scan(d, softplus, io)
    for n, given in (("dD", "D"), ("dz", "z"), ("dbias", "dt_bias"), ("dh0", "h0")):
        assert (got[n] is None) == (d[given] is None)
    for n, t in got.items():
        if t is not None:
            ref.close(n, t, *want[n])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,G,N", [
    (1, 1, 1, 1, 1), (2, 7, 32, 1, 16), (1, 8, 33, 1, 16), (2, 9, 31, 1, 16), (1, 64, 40, 1, 16), (3, 65, 64, 2, 16),
    (1, 130, 96, 1, 16), (2, 40, 24, 4, 4), (1, 77, 10, 5, 8), (2, 50, 12, 1, 24), (1, 30, 36, 3, 64),
    (1, 21, 8, 1, 128), (2, 19, 6, 2, 7), (1, 33, 3, 1, 2), (1, 15, 5, 1, 127), (1, 600, 4, 1, 16)])
def test_forward_and_gradients(B, T, C, G, N, io):
    check(make(B, T, C, G, N, io, seed=T + C, z=T % 2 == 1, state=C % 2 == 0, strided=T % 3 == 0), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("z,state,params,softplus", [
    (False, False, False, False), (True, False, False, True), (False, True, True, True), (True, True, True, False)])
def test_what_may_be_left_out(z, state, params, softplus, io):
    d = make(2, 41, 48, 2, 16, io, seed=11, z=z, state=state, params=params, strided=True)
    if not softplus:    # the steps themselves, 0 to 0.4, whatever the bias (negative ones overflow 64 bits, too)
        bias = 0 if d["dt_bias"] is None else d["dt_bias"]
        d["dt"] = (d["dt"].float().abs() * 0.1 - bias).to(d["dt"].dtype)
    check(d, io, softplus)


@pytest.mark.parametrize("steps", [(1e-6, 1e-5), (0.5, 8.0)])
def test_long_and_short_memories(steps):
    check(make(1, 200, 32, 1, 16, "f32", seed=4, steps=steps), "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 1000])
def test_sequences_in_segments(splits, io):
    """The join of segments adds a few roundings to a state for each of them; the bounds count several for each token."""
    check(make(2, 203, 40, 2, 16, io, seed=splits, steps=(1e-3, 0.5)), io, seq_splits=splits)
    check(make(1, 90, 70, 1, 16, io, seed=splits + 1, state=False), io, seq_splits=splits)
    check(make(1, 65, 9, 1, 11, io, seed=splits + 2, strided=True), io, seq_splits=splits)


@pytest.mark.parametrize("B,T,C,G,N", [(1, 1500, 32, 1, 16), (2, 700, 19, 1, 16), (1, 900, 16, 2, 8), (1, 520, 6, 1, 96)])
def test_few_channels(B, T, C, G, N):
    """What is cut by the rule."""
    check(make(B, T, C, G, N, "f32", seed=T, state=False), "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C,G,N", [(64, 1, 16), (40, 5, 16), (96, 2, 12), (33, 1, 16)])
def test_alignment(C, G, N, io):
    """Each input on its own off 16 bytes: by its pointer, and by its rows."""
    d = make(2, 37, C, G, N, io, seed=C)
    for n in ("u", "dt", "z", "Bm", "Cm", "do"):
        t = d[n].flatten(2)
        for lo, wide in ((1, 1), (0, 3), (8, 8)):
            rows = torch.zeros(*t.shape[:2], t.shape[2] + lo + 8 * wide, dtype=t.dtype)
            rows[..., lo:lo + t.shape[2]] = t
            check({**d, n: rows[..., lo:lo + t.shape[2]].unflatten(-1, d[n].shape[2:])}, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C,N", [(64, 16), (19, 16)])
def test_time_major_inputs(C, N, io):
    """Tensors laid out [T, B, C], and batch entries whose distance is no multiple of a token's."""
    d = make(3, 37, C, 1, N, io, seed=C)
    for n in ("u", "dt", "z", "Bm", "Cm", "do"):
        d[n] = d[n].transpose(0, 1).contiguous().transpose(0, 1)
    check(d, io)
    for n in ("u", "z", "Bm", "do"):
        t = d[n]
        w = t[0, 0].numel()
        flat = torch.zeros(3 * (37 * w + 8), dtype=t.dtype)
        v = flat.as_strided((3, 37, w), (37 * w + 8, w, 1))
        v.copy_(t.flatten(2))
        d[n] = v.unflatten(-1, t.shape[2:])
    check(d, io)


def test_more_than_32_bits_of_elements():
    """Outputs and pages past 2^31 elements, against the same on their own."""
    from chunkwise_recurrent_prefill_gb300 import last_device_status, ssm_fwd, ssm_step
    T, C, N = (1 << 20) + 11, 2080, 8
    g = torch.Generator("cuda").manual_seed(1)
    u = torch.empty(1, T, C, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    dt = torch.empty_like(u).normal_(generator=g)
    Bm, Cm = (torch.randn(1, T, 1, N, device="cuda", generator=g).bfloat16() for _ in range(2))
    A = -torch.rand(C, N, device="cuda", generator=g) - 0.5
    o, hT = ssm_fwd(u, dt, A, Bm, Cm, return_state=True)
    cut = T - 1000
    part = [t[:, :cut] for t in (u, dt)] + [A] + [t[:, :cut] for t in (Bm, Cm)]
    h = ssm_fwd(*part, return_state=True)[1]
    part = [t[:, cut:].contiguous() for t in (u, dt)] + [A] + [t[:, cut:].contiguous() for t in (Bm, Cm)]
    o2, h2 = ssm_fwd(*part, h0=h, return_state=True)
    # the same operations in the same order, but for where a chunk ends
    assert torch.allclose(o[:, cut:].float(), o2.float(), rtol=2.0 ** -7, atol=1e-4)
    assert torch.allclose(hT, h2, rtol=1e-5, atol=1e-6)
    del o, u, dt
    S = torch.empty(40000, 4096, 16, device="cuda")
    few = torch.randn(2, 4096, 16, device="cuda", generator=g)
    S[39999], S[35000] = few[0], few[1]
    x = torch.randn(2, 4096, device="cuda", generator=g)
    b = torch.randn(2, 1, 16, device="cuda", generator=g)
    A = -torch.rand(4096, 16, device="cuda", generator=g)
    o = ssm_step(x, x, A, b, b, S, torch.tensor([39999, 35000], dtype=torch.int32, device="cuda"))
    o2 = ssm_step(x, x, A, b, b, few)
    assert torch.equal(o, o2) and torch.equal(S[39999], few[0]) and torch.equal(S[35000], few[1])
    assert last_device_status() == 0


def test_steps_of_zero_keep_the_state():
    """Bit for bit, whatever A is."""
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd, ssm_step
    t = {k: ref.gpu(v) for k, v in make(2, 50, 40, 1, 16, "f32", seed=3).items()}
    dt = torch.zeros_like(t["dt"])
    A = t["A"] * torch.logspace(-6, 6, 40, device="cuda")[:, None]
    A[3, 2] = -3e38
    hT = ssm_fwd(t["u"], dt, A, t["Bm"], t["Cm"], h0=t["h0"], softplus=False, return_state=True)[1]
    assert torch.equal(hT, t["h0"])
    S = t["h0"].clone()
    ssm_step(t["u"][:, 0], dt[:, 0], A, t["Bm"][:, 0], t["Cm"][:, 0], S, softplus=False)
    assert torch.equal(S, t["h0"])


def test_no_tokens_and_no_channels():
    from chunkwise_recurrent_prefill_gb300 import ssm_bwd, ssm_fwd
    d = {n: ref.gpu(v) for n, v in make(2, 0, 8, 1, 16, "f32").items()}
    got = call(d)
    assert torch.equal(got["hT"], d["h0"]) and torch.equal(got["dh0"], d["dhT"]) and got["o"].shape == (2, 0, 8)
    for n in ("dA", "dD", "dbias"):
        assert not got[n].any()
    a = [torch.zeros(2, 5, 0, device="cuda")] * 2 + [torch.zeros(0, 4, device="cuda")] + \
        [torch.zeros(2, 5, 1, 4, device="cuda")] * 2
    o, hT = ssm_fwd(*a, return_state=True)
    assert o.numel() == 0 and hT.shape == (2, 0, 4)
    dBm = ssm_bwd(o, *a)[3]
    assert dBm.shape == (2, 5, 1, 4) and not dBm.any()


def test_pieces_are_the_whole():
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd
    t = {n: ref.gpu(v) for n, v in make(2, 150, 40, 1, 16, "f32", seed=8, state=False).items()}
    k = dict(D=t["D"], dt_bias=t["dt_bias"], return_state=True)
    whole, end = ssm_fwd(t["u"], t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], **k)
    h, parts = None, []
    for lo, hi in ((0, 8), (8, 72), (72, 73), (73, 150)):
        s = slice(lo, hi)
        o, h = ssm_fwd(*(t[n][:, s] if n != "A" else t[n] for n in ("u", "dt", "A", "Bm", "Cm")), z=t["z"][:, s], h0=h, **k)
        parts.append(o)
    # the same operations in the same order, but for where a chunk ends
    assert torch.allclose(torch.cat(parts, 1), whole, rtol=1e-5, atol=1e-6)
    assert torch.allclose(h, end, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C,G,N", [(40, 1, 16), (9, 3, 4), (256, 1, 16), (6, 1, 7), (5, 1, 128), (33, 1, 64)])
def test_steps(C, G, N, io):
    """Steps on pages against the whole sequence; empty rows and other pages stay as they were."""
    from chunkwise_recurrent_prefill_gb300 import last_device_status, ssm_step
    R, P, n = 5, 9, 6
    d = make(R, n, C, G, N, io, seed=C, strided=True, state=False)
    pool = ref.draw(torch.Generator().manual_seed(1), P, C, N)
    slots, live = torch.tensor([7, -1, 0, 3, -5], dtype=torch.int32), [0, 2, 3]
    at = slots[live].long()
    sub = {k: (v if k in ("A", "D", "dt_bias") or v is None else v[live]) for k, v in d.items()}
    want = ref.scan({**sub, "h0": pool[at]}, io=io, back=False)
    t = {k: ref.gpu(v) for k, v in d.items()}
    S, sl = pool.cuda(), slots.cuda()
    out = torch.stack([ssm_step(t["u"][:, i], t["dt"][:, i], t["A"], t["Bm"][:, i], t["Cm"][:, i], S, sl, D=t["D"],
                                z=t["z"][:, i], dt_bias=t["dt_bias"]) for i in range(n)], 1)
    assert last_device_status() == 0
    ref.close("o", out[live], *want["o"])
    ref.close("S", S[at.cuda()], *want["hT"])
    assert not out[[1, 4]].any()
    rest = [i for i in range(P) if i not in (7, 0, 3)]
    assert torch.equal(S[rest].cpu(), pool[rest])


def test_a_slot_past_the_pool_is_reported():
    from chunkwise_recurrent_prefill_gb300 import last_device_status, ssm_step
    t = {k: ref.gpu(v) for k, v in make(2, 1, 24, 1, 16, "f32").items()}
    S = torch.randn(3, 24, 16, device="cuda")
    before = S.clone()
    o = ssm_step(t["u"][:, 0], t["dt"][:, 0], t["A"], t["Bm"][:, 0], t["Cm"][:, 0], S,
                 torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    assert last_device_status() == 12 and last_device_status() == 0
    assert not o[0].any() and torch.equal(S[[0, 2]], before[[0, 2]]) and not torch.equal(S[1], before[1])


def test_what_is_not_finite_stays_where_it_belongs():
    t = {k: ref.gpu(v) for k, v in make(2, 100, 40, 2, 16, "f32", seed=2).items()}
    clean = call(t)
    t["u"][0, 50, 7] = float("nan")
    got = call(t)
    bad = torch.zeros(2, 100, 40, dtype=torch.bool, device="cuda")
    bad[0, 50:, 7] = True
    assert torch.equal(got["o"][~bad], clean["o"][~bad]) and got["o"][bad].isnan().all()
    assert got["hT"][0, 7].isnan().all()
    ok = torch.ones(2, 40, dtype=torch.bool, device="cuda")
    ok[0, 7] = False
    assert torch.equal(got["hT"][ok], clean["hT"][ok])
    # the gradient of dt reads the states; du does not
    for n in ("ddt", "du"):
        keep = torch.ones_like(bad)
        keep[0, :, 7] = False
        assert torch.equal(got[n][keep], clean[n][keep]), n
    # other groups' sums and earlier tokens'
    assert torch.equal(got["dC"][1], clean["dC"][1]) and torch.equal(got["dC"][0, :50], clean["dC"][0, :50])
    assert torch.equal(got["dC"][0, :, 1], clean["dC"][0, :, 1])


def test_gradient_against_differences():
    d = make(1, 19, 6, 2, 4, "f32", seed=5)
    got = call({n: ref.gpu(v) for n, v in d.items()})
    base = {n: None if v is None else v.double() for n, v in d.items()}
    gen = torch.Generator().manual_seed(6)
    names = dict(u="du", dt="ddt", A="dA", Bm="dB", Cm="dC", D="dD", z="dz", dt_bias="dbias", h0="dh0")
    for n, gname in names.items():
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)

        def loss(e):
            r = ref.scan({**base, n: base[n] + e * v}, back=False)
            return ((r["o"][0] * base["do"]).sum() + (r["hT"][0] * base["dhT"]).sum()).item()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = got[gname].cpu().double() * v
        # the difference is off by h^2 of the third derivative, the gradient by 1e-6 of its terms
        assert abs(terms.sum().item() - want) <= 2e-5 * terms.abs().sum().item() + 1e-6, n


def test_streams_and_graphs():
    from chunkwise_recurrent_prefill_gb300 import ssm_bwd, ssm_fwd, ssm_step, ssm_workspace_size
    t = {n: ref.gpu(v) for n, v in make(2, 100, 64, 1, 16, "bf16", seed=9).items()}
    a = (t["u"], t["dt"], t["A"], t["Bm"], t["Cm"])
    k = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], h0=t["h0"])
    one = (t["u"][:, 0], t["dt"][:, 0], t["A"], t["Bm"][:, 0], t["Cm"][:, 0])
    S = t["h0"].clone()
    want = (*ssm_fwd(*a, return_state=True, **k), *ssm_bwd(t["do"], *a, dhT=t["dhT"], **k), ssm_step(*one, S.clone()))
    ws = torch.empty(max(ssm_workspace_size(*a, z=t["z"], backward=True), 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*ssm_fwd(*a, return_state=True, stream=side, **k), *ssm_bwd(t["do"], *a, dhT=t["dhT"], stream=side, **k),
           ssm_step(*one, S.clone(), stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = (*ssm_fwd(*a, return_state=True, **k), *ssm_bwd(t["do"], *a, dhT=t["dhT"], workspace=ws, **k),
               ssm_step(*one, S))
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_a_workspace_that_is_too_small():
    from chunkwise_recurrent_prefill_gb300 import GLAError, ssm_bwd, ssm_workspace_size
    t = {n: ref.gpu(v) for n, v in make(1, 50, 64, 1, 16, "f32").items()}
    a = (t["u"], t["dt"], t["A"], t["Bm"], t["Cm"])
    assert ssm_workspace_size(*a, backward=True) > 4096
    with pytest.raises(GLAError, match="WORKSPACE"):
        ssm_bwd(t["do"], *a, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
