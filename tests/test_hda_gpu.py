"""Decay attention (hda_fwd, hda_bwd, hda_step) against its 64-bit form; the bounds are derived
in hda_ref.py."""
import pytest
import torch

import hda_ref as ref

pytestmark = pytest.mark.gpu

# every path that can run the case
SHAPES = [
    # B, T, H, Hq, Hk, Hv, Dk, Dv
    (2, 1, 3, 3, 3, 3, 64, 64),
    (1, 2, 4, 4, 2, 1, 128, 64),
    (2, 63, 2, 1, 2, 2, 64, 128),
    (1, 64, 3, 3, 1, 3, 128, 128),
    (1, 65, 2, 2, 2, 2, 128, 128),
    (3, 130, 4, 2, 1, 4, 64, 64),
    (1, 331, 2, 2, 2, 2, 128, 128),
    (2, 200, 6, 3, 2, 6, 64, 128),
]
ODD_DIMS = [(2, 37, 2, 2, 1, 2, 8, 16), (1, 70, 3, 1, 3, 3, 96, 40), (1, 45, 1, 1, 1, 1, 256, 200)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _gpu(x):
    return {n: ref.to_gpu(t) for n, t in x.items()}


def _paths(g, path_names=("exact", "tc")):
    from chunkwise_recurrent_prefill_gb300 import hda_path_for
    return [p for p in path_names if hda_path_for(g["q"], g["k"], g["v"], g["decay"], p) == p]


def _status_ok():
    from chunkwise_recurrent_prefill_gb300 import last_device_status
    assert last_device_status() == 0


def _check_forward(x, path, splits=0):
    from chunkwise_recurrent_prefill_gb300 import hda_fwd
    g = _gpu(x)
    o, hT = hda_fwd(g["q"], g["k"], g["v"], g["decay"], x["scale"], g.get("h0"), return_state=True,
                    path=path, seq_splits=splits)
    _status_ok()
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x.get("h0"))
    want = ref.forward(*a)
    absolute = ref.forward(*[t.abs() if isinstance(t, torch.Tensor) and i != 3 else t
                             for i, t in enumerate(a)])
    T, Dk = x["q"].shape[1], x["q"].shape[3]
    ref.check(f"o {path}", o, want[0], absolute[0], T, Dk, path)
    ref.check(f"hT {path}", hT, want[1], absolute[1], T, Dk, path, state=True)


def _check_backward(x, path, splits=0):
    from chunkwise_recurrent_prefill_gb300 import hda_bwd
    g = _gpu(x)
    got = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g.get("h0"),
                  g.get("dhT"), path=path, seq_splits=splits)
    _status_ok()
    a = (x["do"], x["q"], x["k"], x["v"], x["decay"], x["scale"], x.get("h0"), x.get("dhT"))
    want = ref.backward(*a)
    absolute = ref.backward(*[t.abs() if isinstance(t, torch.Tensor) and i != 4 else t
                              for i, t in enumerate(a)])
    T, D = x["q"].shape[1], max(x["q"].shape[3], x["v"].shape[3])
    for n, got_n, want_n, abs_n in zip(("dq", "dk", "dv"), got, want, absolute):
        ref.check(f"{n} {path}", got_n, want_n, abs_n, T, D, path)
    if x.get("h0") is None:
        assert got[3] is None
    else:
        ref.check(f"dh0 {path}", got[3], want[3], absolute[3], T, D, path, state=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES + ODD_DIMS)
def test_forward_and_gradients(shape, io):
    x = ref.inputs(*shape, io=io, seed=sum(shape), strided=True)
    for path in _paths(_gpu(x)):
        _check_forward(x, path)
        _check_backward(x, path)


@pytest.mark.parametrize("shape", [(1, 200, 2, 2, 2, 2, 128, 128), (2, 77, 2, 2, 1, 2, 64, 64)])
def test_without_states(shape):
    x = ref.inputs(*shape, io="bf16", seed=5)
    del x["h0"], x["dhT"]
    for path in _paths(_gpu(x)):
        _check_forward(x, path)
        _check_backward(x, path)


@pytest.mark.parametrize("decay", [[0.0, -1e-6], [-20.0, -0.7], [-200.0, float("-inf")],
                                   [0.01, -88.0]])
def test_decays_of_every_strength(decay):
    """No decay, decays that a chunk's end no longer feels, none left at all, and growth."""
    x = ref.inputs(1, 150, 2, 2, 2, 2, 128, 128, "bf16", seed=8, decay=decay)
    for path in _paths(_gpu(x)):
        _check_forward(x, path)
        _check_backward(x, path)


def test_infinite_decay_keeps_the_token_alone():
    from chunkwise_recurrent_prefill_gb300 import hda_fwd
    x = _gpu(ref.inputs(1, 5, 1, 1, 1, 1, 16, 16, "f32", seed=9, decay=[float("-inf")]))
    _, hT = hda_fwd(x["q"], x["k"], x["v"], x["decay"], 1.0, x["h0"], return_state=True)
    assert torch.equal(hT[0, 0], x["k"][0, 4, 0][:, None] * x["v"][0, 4, 0][None, :])


@pytest.mark.parametrize("splits", [0, 1, 2, 5, 200])
@pytest.mark.parametrize("dims", [(64, 64), (128, 40), (24, 200), (200, 64)])
def test_sequence_splits_token_by_token(splits, dims):
    """Segments of whole tiles of 16 tokens, the last one shorter; 0: by the rule, which gives one
    head's 777 tokens several."""
    x = ref.inputs(1, 777, 2, 2, 1, 1, dims[0], dims[1], io="f32", seed=splits, decay=[-0.02, -3.0])
    _check_forward(x, "exact", splits)
    _check_backward(x, "exact", splits)


@pytest.mark.parametrize("splits", [1, 2, 3, 7])
def test_sequence_splits(splits):
    x = ref.inputs(1, 64 * 7 + 5, 2, 1, 2, 2, 128, 64, "bf16", seed=10)
    if "tc" in _paths(_gpu(x)):
        _check_forward(x, "tc", splits)
        _check_backward(x, "tc", splits)


@pytest.mark.parametrize("path", ["exact", "tc"])
def test_nothing_leaks_across_tokens_heads_or_entries(path):
    """NaN and infinity at a token touch that head's later outputs, and the gradients of its
    earlier tokens, alone."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd
    x = ref.inputs(2, 150, 2, 2, 2, 2, 128, 128, "bf16", seed=11)
    g = _gpu(x)
    if path not in _paths(g):
        pytest.skip("path not available")
    run = lambda: hda_fwd(g["q"], g["k"], g["v"], g["decay"], 1.0, path=path)[0]  # noqa: E731
    clean = run()
    back = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], 1.0, path=path)
    for n, value in (("k", float("nan")), ("v", float("inf"))):
        kept = g[n].clone()
        g[n][1, 100, 1] = value
        dirty = run()
        assert torch.equal(dirty[0], clean[0]) and torch.equal(dirty[1, :, 0], clean[1, :, 0])
        if path == "exact":
            assert torch.equal(dirty[1, :100, 1], clean[1, :100, 1])
        else:   # a chunk's products see all its tokens: whole chunks before it are untouched
            assert torch.equal(dirty[1, :64, 1], clean[1, :64, 1])
        assert not torch.isfinite(dirty[1, 100:, 1].float()).all()
        g[n] = kept
    g["do"][1, 20, 1] = float("nan")
    dq, dk, dv, _ = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], 1.0, path=path)
    for d, c in zip((dq, dk, dv), back):
        assert torch.equal(d[0], c[0]) and torch.equal(d[1, :, 0], c[1, :, 0])
    first = 21 if path == "exact" else 64
    assert torch.equal(dk[1, first:, 1], back[1][1, first:, 1])
    _status_ok()


def test_gradients_against_differences():
    """<gradient, direction> of the fp32 kernels against central differences of the 64-bit
    forward (exact: the loss is linear in each argument)."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd
    x = ref.inputs(2, 40, 4, 2, 4, 1, 64, 32, "f32", seed=12)
    g = _gpu(x)
    grads = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], g["dhT"])
    args = {n: x[n].double() for n in ("q", "k", "v", "h0")}

    def loss(sign, n, d):
        a = {**args, n: args[n] + sign * d}
        o, hT = ref.forward(a["q"], a["k"], a["v"], x["decay"], x["scale"], a["h0"])
        return (o * x["do"].double()).sum() + (hT * x["dhT"].double()).sum()

    gen = torch.Generator("cpu").manual_seed(4)
    for n, got in zip(("q", "k", "v", "h0"), grads):
        d = torch.randn(args[n].shape, generator=gen, dtype=torch.float64)
        diff = (loss(1, n, d) - loss(-1, n, d)) / 2
        dot = (got.cpu().double() * d).sum()
        # each component is within K u of its absolute sum; 1e-4 of the norm product is far above
        assert abs(dot - diff) <= 1e-4 * got.double().norm().item() * d.norm()


def test_repeated_calls_give_the_same_bits():
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd
    g = _gpu(ref.inputs(1, 1000, 4, 2, 1, 4, 128, 128, "bf16", seed=13))
    a = (g["q"], g["k"], g["v"], g["decay"], 0.1, g["h0"])
    one, two = hda_fwd(*a, return_state=True), hda_fwd(*a, return_state=True)
    assert all(torch.equal(p, r) for p, r in zip(one, two))
    one, two = hda_bwd(g["do"], *a, g["dhT"]), hda_bwd(g["do"], *a, g["dhT"])
    assert all(torch.equal(p, r) for p, r in zip(one, two))


def test_state_carries_over_a_cut():
    """[0, T) in one call, and [0, c) then [c, T) from the returned state."""
    from chunkwise_recurrent_prefill_gb300 import hda_fwd
    x = ref.inputs(1, 500, 2, 2, 2, 2, 128, 128, "bf16", seed=14)
    g = _gpu(x)
    part = lambda n, a, b: g[n][:, a:b]  # noqa: E731  (a view: strided batch)
    o1, h1 = hda_fwd(*(part(n, 0, 131) for n in "qkv"), g["decay"], x["scale"], g["h0"],
                     return_state=True)
    o2, h2 = hda_fwd(*(part(n, 131, 500) for n in "qkv"), g["decay"], x["scale"], h1,
                     return_state=True)
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"])
    want = ref.forward(*a)
    absolute = ref.forward(*[t.abs() if isinstance(t, torch.Tensor) and i != 3 else t
                             for i, t in enumerate(a)])
    path = "tc" if "tc" in _paths(g) else "exact"
    ref.check("o", torch.cat([o1, o2], 1), want[0], absolute[0], 500, 128, path)
    ref.check("hT", h2, want[1], absolute[1], 500, 128, path, state=True)


def test_no_tokens_and_no_batch():
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd
    g = _gpu(ref.inputs(2, 0, 3, 3, 3, 1, 64, 64, "bf16", seed=15))
    a = (g["q"], g["k"], g["v"], g["decay"], 1.0)
    o, hT = hda_fwd(*a, g["h0"], return_state=True)
    assert o.shape == (2, 0, 3, 64) and torch.equal(hT, g["h0"])
    _, hT = hda_fwd(*a, return_state=True)
    assert not hT.any()
    dq, _, _, dh0 = hda_bwd(g["do"], *a, g["h0"], g["dhT"])
    assert dq.numel() == 0 and torch.equal(dh0, g["dhT"])
    g = _gpu(ref.inputs(0, 70, 3, 3, 3, 1, 64, 64, "bf16", seed=15))
    o, hT = hda_fwd(g["q"], g["k"], g["v"], g["decay"], 1.0, g["h0"], return_state=True)
    assert o.numel() == 0 and hT.numel() == 0


def test_other_stream_and_caller_workspace():
    """A call on a side stream with a caller's workspace, captured in a graph and replayed."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd, hda_workspace_size
    g = _gpu(ref.inputs(1, 900, 2, 1, 2, 2, 128, 128, "bf16", seed=16))
    a = (g["q"], g["k"], g["v"], g["decay"], 0.1, g["h0"])
    n = max(hda_workspace_size(*a[:4]), hda_workspace_size(*a[:4], backward=True), 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want_o, want_h = hda_fwd(*a, return_state=True)
    want_g = hda_bwd(g["do"], *a, g["dhT"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hda_fwd(*a, return_state=True, workspace=ws)
        hda_bwd(g["do"], *a, g["dhT"], workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, hT = hda_fwd(*a, return_state=True, workspace=ws)
        grads = hda_bwd(g["do"], *a, g["dhT"], workspace=ws)
    for t in (o, hT) + tuple(grads):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    _status_ok()
    assert torch.equal(o, want_o) and torch.equal(hT, want_h)
    assert all(torch.equal(p, r) for p, r in zip(grads, want_g))


def test_outputs_on_a_given_stream():
    """A call with ``stream=`` does not take memory for its outputs that work still pending on the
    current stream writes to."""
    from chunkwise_recurrent_prefill_gb300 import group_norm_fwd, hda_fwd
    g = _gpu(ref.inputs(1, 700, 2, 2, 2, 2, 128, 128, "bf16", seed=19))
    a = (g["q"], g["k"], g["v"], g["decay"], 0.1)
    want, want_h = hda_fwd(*a, return_state=True)
    want_y = group_norm_fwd(want.view(700, 256), 2)[0]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = [torch.empty_like(t) for t in (want, want_h, want_y) for _ in range(4)]
    torch.cuda._sleep(20_000_000)
    for t in held:
        t.fill_(float("nan"))
    del held, t
    o, hT = hda_fwd(*a, return_state=True, stream=s)
    y = group_norm_fwd(o.view(700, 256), 2, stream=s)[0]
    torch.cuda.synchronize()
    _status_ok()
    assert torch.equal(o, want) and torch.equal(hT, want_h) and torch.equal(y, want_y)


# ---------------------------------------------------------------- single tokens
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("R,P,H,Hq,Hk,Hv,Dk,Dv", [
    (1, 1, 1, 1, 1, 1, 64, 64), (5, 9, 4, 2, 1, 4, 128, 128), (3, 3, 2, 2, 2, 1, 96, 132),
    (2, 4, 3, 1, 3, 3, 1, 4), (2, 2, 1, 1, 1, 1, 200, 260), (40, 50, 2, 2, 2, 2, 64, 128)])
def test_step(io, R, P, H, Hq, Hk, Hv, Dk, Dv):
    from chunkwise_recurrent_prefill_gb300 import hda_step
    x = ref.inputs(R, 1, H, Hq, Hk, Hv, Dk, Dv, io, seed=R + Dk)
    gen = torch.Generator("cpu").manual_seed(R)
    pool = torch.randn(P, H, Dk, Dv, generator=gen)
    slots = torch.randperm(P, generator=gen)[:R].to(torch.int32)
    if R > 2:
        slots[1] = -1
    g = _gpu(x)
    S = pool.cuda()
    o = hda_step(g["q"][:, 0], g["k"][:, 0], g["v"][:, 0], g["decay"], x["scale"], S, slots.cuda())
    _status_ok()
    live = slots >= 0
    at = slots[live].long()
    a = [x[n][live] for n in "qkv"] + [x["decay"], x["scale"], pool[at]]
    want = ref.forward(*a)
    absolute = ref.forward(*[t.abs() if isinstance(t, torch.Tensor) and i != 3 else t
                             for i, t in enumerate(a)])
    ref.check("o", o[live.cuda()][:, None], want[0], absolute[0], 1, Dk)
    ref.check("S", S.cpu()[at], want[1], absolute[1], 1, Dk, state=True)
    assert not o[~live.cuda()].any()
    rest = torch.ones(P, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(S.cpu()[rest], pool[rest])        # no other page is touched


def test_step_continues_a_prompt():
    from chunkwise_recurrent_prefill_gb300 import hda_fwd, hda_step
    x = ref.inputs(2, 130, 4, 4, 2, 4, 128, 128, "bf16", seed=21)
    g = _gpu(x)
    _, S = hda_fwd(*(g[n][:, :126] for n in "qkv"), g["decay"], x["scale"], g["h0"],
                   return_state=True)
    outs = [hda_step(*(g[n][:, t] for n in "qkv"), g["decay"], x["scale"], S)
            for t in range(126, 130)]
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"])
    want = ref.forward(*a)
    absolute = ref.forward(*[t.abs() if isinstance(t, torch.Tensor) and i != 3 else t
                             for i, t in enumerate(a)])
    path = "tc" if "tc" in _paths(g) else "exact"
    ref.check("o", torch.stack(outs, 1), want[0][:, 126:], absolute[0][:, 126:], 130, 128, path,
              state=True)
    ref.check("S", S, want[1], absolute[1], 130, 128, path, state=True)


def test_step_reports_a_slot_out_of_range():
    from chunkwise_recurrent_prefill_gb300 import hda_step, last_device_status
    x = _gpu(ref.inputs(2, 1, 1, 1, 1, 1, 64, 64, "bf16", seed=22))
    S = torch.ones(3, 1, 64, 64, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    o = hda_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["decay"], 1.0, S, slots)
    assert last_device_status() == 12 and last_device_status() == 0
    assert not o[0].any() and o[1].any()
    assert torch.equal(S[[0, 2]], torch.ones_like(S[[0, 2]]))


# ---------------------------------------------------------------- refusals
def test_refusals():
    from chunkwise_recurrent_prefill_gb300 import GLAError, hda_bwd, hda_fwd, hda_step
    x = _gpu(ref.inputs(1, 70, 4, 4, 2, 4, 128, 128, "bf16", seed=30))
    q, k, v, d = x["q"], x["k"], x["v"], x["decay"]
    with pytest.raises(TypeError):
        hda_fwd(q.half(), k.half(), v.half(), d, 1.0)
    with pytest.raises(TypeError):
        hda_fwd(q, k.float(), v, d, 1.0)
    with pytest.raises(TypeError):
        hda_fwd(q, k, v, d.double(), 1.0)
    with pytest.raises(ValueError):
        hda_fwd(q, k[:, :-1], v, d, 1.0)                       # other lengths
    with pytest.raises(ValueError):
        hda_fwd(q.transpose(2, 3), k.transpose(2, 3), v, d, 1.0)
    with pytest.raises(ValueError):
        hda_fwd(q[:, :1].expand(-1, 70, -1, -1), k, v, d, 1.0)  # a stride of zero
    with pytest.raises(ValueError):
        hda_fwd(q.cpu(), k.cpu(), v.cpu(), d.cpu(), 1.0)
    with pytest.raises(ValueError):
        hda_fwd(q, k, v, d, 1.0, x["h0"][:, :2])
    with pytest.raises(GLAError, match="BAD_SHAPE"):
        hda_fwd(q[:, :, :3].contiguous(), k, v, d, 1.0)        # 3 heads do not divide 4
    with pytest.raises(GLAError, match="UNSUPPORTED_DIM"):
        hda_fwd(q.repeat(1, 1, 1, 3), k.repeat(1, 1, 1, 3), v, d, 1.0)   # 384 wide
    with pytest.raises(GLAError, match="UNSUPPORTED_DIM"):
        hda_fwd(q.float(), k.float(), v.float(), d, 1.0, path="tc")
    with pytest.raises(GLAError, match="ALIAS"):
        hda_fwd(q, k, v, d, 1.0, x["h0"], hT=x["h0"])
    with pytest.raises(GLAError, match="ALIAS"):
        hda_fwd(q, k, v, d, 1.0, o=v)
    with pytest.raises(GLAError, match="BAD_OPTION"):
        hda_fwd(q, k, v, d, 1.0, seq_splits=-1)
    with pytest.raises(GLAError, match="WORKSPACE"):
        hda_bwd(x["do"], q, k, v, d, 1.0, workspace=torch.empty(16, device="cuda"))
    with pytest.raises(ValueError):
        hda_bwd(x["do"][:, :, :2], q, k, v, d, 1.0)
    S = torch.zeros(2, 4, 128, 128, device="cuda")
    with pytest.raises(TypeError):
        hda_step(q[:, 0], k[:, 0], v[:, 0], d, 1.0, S, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        hda_step(q[:, 0], k[:, 0], v[:, 0], d, 1.0, S[:, :2])
    with pytest.raises(GLAError, match="BAD_SHAPE"):
        hda_step(q[0], k[0], v[0], d, 1.0, S)                  # 70 rows, 2 pages, no slots
