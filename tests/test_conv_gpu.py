"""Short causal convolution against its 64-bit form (bounds: layer_ref.py)."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def make(B, T, C, W, io, seed, state=True, bias=True, strided=False):
    g = torch.Generator().manual_seed(seed)

    def rows():
        if strided:
            return ref.draw(g, B, T, 3 * C + 1, io=io)[..., C:2 * C]
        return ref.draw(g, B, T, C, io=io)

    return dict(x=rows(), dy=rows(), w=ref.draw(g, C, W, std=W ** -0.5),
                bias=ref.draw(g, C, std=0.2) if bias else None,
                s0=ref.draw(g, B, W - 1, C, io=io) if state else None,
                dsT=ref.draw(g, B, W - 1, C, io=io) if state else None)


def check(d, act, io):
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd, last_device_status
    x, dy, w, bias, s0, dsT = (ref.gpu(d[n]) for n in ("x", "dy", "w", "bias", "s0", "dsT"))
    y, sT = conv_fwd(x, w, bias, s0, act=act, return_state=True)
    dx, dw, db, ds0 = conv_bwd(dy, x, w, bias, s0, dsT, act=act)
    assert last_device_status() == 0
    want = ref.conv(d["x"], d["w"], d["bias"], d["s0"], d["dy"], d["dsT"], act, io)
    got = dict(y=y, sT=sT, dx=dx, dw=dw, db=db, ds0=ds0)
    assert (db is None) == (d["bias"] is None) and (ds0 is None) == (d["s0"] is None)
    for n, t in got.items():
        if t is not None:
            ref.close(n, t, *want[n])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
def test_widths(W, act, io):
    check(make(2, 37, 40, W, io, seed=W), act, io)
    check(make(2, 13, 9, W, io, seed=W, strided=True, state=False), act, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,C,W", [
    (1, 1, 1, 4), (1, 1, 8, 2), (3, 2, 24, 4), (2, 3, 16, 8), (1, 7, 5, 8), (2, 64, 8, 4), (2, 65, 16, 4),
    (1, 300, 264, 4), (5, 129, 33, 3), (1, 2049, 72, 4), (70, 5, 8, 4), (1, 515, 1024, 4), (3, 8, 2052, 5)])
def test_sizes(B, T, C, W, io):
    check(make(B, T, C, W, io, seed=B + T + C, state=T % 2 == 1, bias=C % 2 == 0), "silu", io)
    check(make(B, T, C, W, io, seed=T, strided=True), "silu", io)


def test_no_tokens_and_no_channels():
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd
    w, s0 = torch.randn(16, 4, device="cuda"), torch.randn(2, 3, 16, device="cuda")
    x = torch.empty(2, 0, 16, device="cuda")
    y, sT = conv_fwd(x, w, None, s0, return_state=True)
    assert y.shape == x.shape and torch.equal(sT, s0)
    assert not conv_fwd(x, w, return_state=True)[1].any()
    dx, dw, db, ds0 = conv_bwd(x, x, w, w[:, 0].contiguous(), s0, s0)
    assert dx.shape == x.shape and not dw.any() and not db.any() and torch.equal(ds0, s0)
    y, sT = conv_fwd(torch.empty(2, 5, 0, device="cuda"), torch.empty(0, 4, device="cuda"), return_state=True)
    assert y.numel() == 0 and sT.shape == (2, 3, 0)


def test_pieces_are_the_whole():
    """A sequence cut anywhere, the state handed on, gives the same bits."""
    from chunkwise_recurrent_prefill_gb300 import conv_fwd
    g = torch.Generator().manual_seed(3)
    for io in ("bf16", "f32"):
        x = ref.gpu(ref.draw(g, 2, 100, 48, io=io))
        w, b = ref.gpu(ref.draw(g, 48, 4)), ref.gpu(ref.draw(g, 48))
        whole, end = conv_fwd(x, w, b, act="silu", return_state=True)
        s, parts = None, []
        for lo, hi in ((0, 1), (1, 3), (3, 70), (70, 72), (72, 100)):
            y, s = conv_fwd(x[:, lo:hi], w, b, s, act="silu", return_state=True)
            parts.append(y)
        assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(s, end)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C,W", [(40, 4), (9, 3), (2048, 4), (16, 1), (8, 8)])
def test_steps(C, W, io):
    """Steps on pages give what the whole sequence gives; empty rows and other pages stay as they were."""
    from chunkwise_recurrent_prefill_gb300 import conv_fwd, conv_step, last_device_status
    g = torch.Generator().manual_seed(C + W)
    R, P, n = 5, 9, 12
    x = ref.gpu(ref.draw(g, R, n, 2 * C, io=io))[..., :C]
    w, b = ref.gpu(ref.draw(g, C, W)), ref.gpu(ref.draw(g, C))
    pool = ref.gpu(ref.draw(g, P, W - 1, C, io=io))
    slots = torch.tensor([7, -1, 0, 3, -5], dtype=torch.int32, device="cuda")
    live = [0, 2, 3]
    at = slots[live].long()
    whole, end = conv_fwd(x[live], w, b, pool[at].contiguous(), act="silu", return_state=True)
    before = pool.clone()
    outs = [conv_step(x[:, t], w, pool, slots, b, act="silu") for t in range(n)]
    assert last_device_status() == 0
    out = torch.stack(outs, 1)
    assert torch.equal(out[live], whole) and not out[[1, 4]].any()
    assert torch.equal(pool[at], end)
    rest = [i for i in range(P) if i not in (7, 0, 3)]
    assert torch.equal(pool[rest], before[rest])
    # without slots: row r is page r
    y = conv_step(x[:, 0], w, before, None, b, act="silu")
    assert y.shape == (R, C)


def test_a_slot_past_the_pool_is_reported():
    from chunkwise_recurrent_prefill_gb300 import conv_step, last_device_status
    pool, w = torch.randn(3, 3, 16, device="cuda"), torch.randn(16, 4, device="cuda")
    before = pool.clone()
    x = torch.randn(2, 16, device="cuda")
    y = conv_step(x, w, pool, torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    assert last_device_status() == 12 and last_device_status() == 0
    assert not y[0].any() and torch.equal(pool[[0, 2]], before[[0, 2]]) and torch.equal(pool[1, 2], x[1])


def test_what_is_not_finite_stays_where_it_belongs():
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd
    x = torch.randn(2, 200, 64, device="cuda")
    w, dy = torch.randn(64, 4, device="cuda"), torch.randn(2, 200, 64, device="cuda")
    clean, dclean = conv_fwd(x, w, act="silu")[0], conv_bwd(dy, x, w, act="silu")[0]
    x[0, 70, 5], x[1, 199, 9] = float("nan"), float("inf")
    y, dx = conv_fwd(x, w, act="silu")[0], conv_bwd(dy, x, w, act="silu")[0]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 70:74, 5] = bad[1, 199, 9] = True
    assert torch.equal(y[~bad], clean[~bad]) and y[0, 70:74, 5].isnan().all()
    bad[0, 67:74, 5] = bad[1, 196:, 9] = True
    assert torch.equal(dx[~bad], dclean[~bad])


def test_gradient_against_differences():
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd
    d = make(2, 11, 12, 4, "f32", seed=5)
    t = {n: ref.gpu(v) for n, v in d.items()}
    grads = conv_bwd(t["dy"], t["x"], t["w"], t["bias"], t["s0"], t["dsT"], act="silu")
    base = {n: d[n].double() for n in ("x", "w", "bias", "s0")}
    gen = torch.Generator().manual_seed(6)
    for n, g in zip(("x", "w", "bias", "s0"), grads):
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)

        def loss(e):
            a = {**base, n: base[n] + e * v}
            r = ref.conv(a["x"], a["w"], a["bias"], a["s0"], None, None, "silu", "f32")
            return ((r["y"][0] * d["dy"].double()).sum() + (r["sT"][0] * d["dsT"].double()).sum()).item()

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        got = (g.cpu().double() * v).sum().item()
        # the difference is off by h^2 of the third derivative, the gradient by 1e-6 of its terms
        assert abs(got - want) <= 2e-5 * (g.cpu().double() * v).abs().sum().item() + 1e-6


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C", [64, 19])
def test_time_major_inputs(C, io):
    d = make(3, 37, C, 4, io, seed=C)
    for n in ("x", "dy"):
        d[n] = d[n].transpose(0, 1).contiguous().transpose(0, 1)
    check(d, "silu", io)


def test_more_than_32_bits_of_elements():
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd, conv_step
    T, C = (1 << 20) + 11, 2080
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, T, C, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w = torch.randn(C, 4, device="cuda", generator=g)
    y = conv_fwd(x, w, act="silu")[0]
    cut = T - 1000
    s0 = x[:, cut - 3:cut].contiguous()
    assert torch.equal(y[:, cut:], conv_fwd(x[:, cut:].contiguous(), w, None, s0, act="silu")[0])
    dx = conv_bwd(y, x, w, act="silu")[0]
    dx2 = conv_bwd(y[:, cut:].contiguous(), x[:, cut:].contiguous(), w, None, s0, act="silu")[0]
    assert torch.equal(dx[:, cut:], dx2)
    del x, y, dx
    S = torch.empty(200000, 3, 4096, device="cuda", dtype=torch.bfloat16)
    few = torch.randn(2, 3, 4096, device="cuda", generator=g).bfloat16()
    S[199999], S[180000] = few[0], few[1]
    x, w = torch.randn(2, 4096, device="cuda", generator=g).bfloat16(), torch.randn(4096, 4, device="cuda", generator=g)
    y = conv_step(x, w, S, torch.tensor([199999, 180000], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, conv_step(x, w, few)) and torch.equal(S[199999], few[0]) and torch.equal(S[180000], few[1])


def test_streams_and_graphs():
    """On a stream of its own, with the library's workspace and one of the caller's, and replayed."""
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd, conv_step, conv_workspace_size
    d = {n: ref.gpu(v) for n, v in make(2, 300, 128, 4, "bf16", seed=9).items()}
    args = (d["x"], d["w"], d["bias"], d["s0"])
    pool = d["s0"].clone()
    want = conv_fwd(*args, act="silu")[0], *conv_bwd(d["dy"], *args, d["dsT"], act="silu")
    step = conv_step(d["x"][:, 0], d["w"], pool.clone(), None, d["bias"])
    ws = torch.empty(conv_workspace_size(d["x"], d["w"]), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = conv_fwd(*args, act="silu", stream=side)[0], *conv_bwd(d["dy"], *args, d["dsT"], act="silu", stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = conv_fwd(*args, act="silu")[0], *conv_bwd(d["dy"], *args, d["dsT"], act="silu", workspace=ws)
        out = conv_step(d["x"][:, 0], d["w"], pool, None, d["bias"])
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(out, step)


def test_a_workspace_that_is_too_small():
    from chunkwise_recurrent_prefill_gb300 import GLAError, conv_bwd, conv_workspace_size
    x, w = torch.randn(1, 50, 64, device="cuda"), torch.randn(64, 4, device="cuda")
    n = conv_workspace_size(x, w)
    assert n > 0
    with pytest.raises(GLAError, match="WORKSPACE"):
        conv_bwd(x, x, w, workspace=torch.empty(n - 4, dtype=torch.uint8, device="cuda"))
