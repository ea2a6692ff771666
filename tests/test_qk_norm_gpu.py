"""Norm of queries and keys with their rotation against the 64-bit form (bounds: layer_ref.py)."""
import pytest
import torch

import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def table(P, R):
    f = 10000.0 ** (-torch.arange(R // 2).double() * 2 / max(R, 1))
    a = torch.arange(P).double()[:, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def make(B, T, Hq, Hk, D, R, io="f32", seed=0, norm="rms", weights=True, strided=False, P=None):
    g = torch.Generator().manual_seed(seed)

    def heads(n):
        if not strided:
            return ref.draw(g, B, T, n, D, io=io)
        return ref.draw(g, B, T, n, 2 * D + 1, io=io)[..., 1:D + 1]

    weights = weights and norm != "none"
    P = P or T + 3
    d = dict(q=heads(Hq), k=heads(Hk), dqo=heads(Hq), dko=heads(Hk),
             wq=1 + ref.draw(g, D, std=0.3) if weights else None, wk=1 + ref.draw(g, D, std=0.3) if weights else None)
    d["cos"], d["sin"] = table(P, R) if R else (None, None)
    d["positions"] = torch.randint(0, P, (B, T), generator=g).to(torch.int32)
    return d


def call(t, norm, layout, eps=1e-6, **kw):
    from chunkwise_recurrent_prefill_gb300 import qk_norm_bwd, qk_norm_fwd
    k = dict(cos=t["cos"], sin=t["sin"], positions=t["positions"], norm=norm, layout=layout)
    qo, ko, rq, rk = qk_norm_fwd(t["q"], t["k"], t["wq"], t["wk"], eps=eps, **k)
    return (qo, ko, rq, rk) + qk_norm_bwd(t["dqo"], t["dko"], t["q"], t["k"], rq, rk, t["wq"], t["wk"], **k, **kw)


def check(d, norm, layout, eps=1e-6, status=0):
    from chunkwise_recurrent_prefill_gb300 import last_device_status
    qo, ko, rq, rk, dq, dk, dwq, dwk = call({n: ref.gpu(v) for n, v in d.items()}, norm, layout, eps)
    assert last_device_status() == status
    pos = d["positions"]
    if pos is None:
        pos = torch.arange(d["q"].shape[1]).expand(d["q"].shape[:2])
    for x, go, w, o, r, dx, dw in (("q", "dqo", "wq", qo, rq, dq, dwq), ("k", "dko", "wk", ko, rk, dk, dwk)):
        want = ref.qk(d[x], d[w], d["cos"], d["sin"], pos, norm, layout == "pairs", eps, d[go],
                      None if r is None else r.cpu())
        ref.close(x + "o", o, *want["out"])
        ref.close("d" + x, dx, *want["dx"])
        assert (r is None) == (norm == "none") and (dw is None) == (d[w] is None)
        if r is not None:
            ref.close("r" + x, r, *want["r"])
        if dw is not None:
            ref.close("d" + w, dw, *want["dw"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 32), (128, 128), (128, 0), (80, 80), (80, 20), (96, 64)])
def test_norms_and_layouts(D, R, norm, layout, io):
    check(make(2, 9, 4, 2, D, R, io, seed=D + R, norm=norm), norm, layout)
    check(make(1, 5, 3, 1, D, R, io, seed=R, norm=norm, strided=True, weights=False), norm, layout)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [
    (1, 1, 1, 1, 1, 0), (1, 1, 1, 1, 2, 2), (2, 3, 5, 3, 7, 6), (1, 40, 2, 1, 33, 10), (3, 17, 16, 4, 128, 128),
    (1, 300, 16, 16, 64, 64), (70, 1, 4, 4, 256, 256), (1, 11, 2, 2, 1024, 1024), (1, 9, 2, 2, 1000, 72),
    (2, 5, 1, 1, 192, 96), (1, 7, 6, 2, 48, 48), (1, 6, 2, 1, 512, 256), (1, 4, 3, 0, 64, 64)])
def test_sizes(B, T, Hq, Hk, D, R, io):
    check(make(B, T, Hq, Hk, D, R, io, seed=T + D, strided=T % 2 == 0), "rms", "halves")
    check(make(B, T, Hq, Hk, D, R, io, seed=T + D, strided=T % 2 == 1), "rms", "pairs")


def test_positions_by_index():
    d = make(2, 12, 2, 2, 64, 64, seed=1)
    d["positions"] = None
    check(d, "rms", "halves")


@pytest.mark.parametrize("D", [64, 7])
def test_positions_outside_of_the_table(D):
    """Zeros and a status for those tokens, no part in the sums; the others as ever."""
    d = make(2, 12, 3, 2, D, D // 2 * 2, seed=2, P=30)
    d["positions"][0, 3], d["positions"][1, 0], d["positions"][1, 11] = 30, -1, 2 ** 31 - 1
    check(d, "rms", "halves", status=12)
    d = make(1, 5, 2, 2, D, D // 2 * 2, seed=2, P=4)
    d["positions"] = None           # the fifth token is past the table
    check(d, "l2", "pairs", status=12)


def test_no_tokens():
    d = {n: ref.gpu(v) for n, v in make(2, 0, 4, 2, 64, 64).items()}
    qo, ko, rq, rk, dq, dk, dwq, dwk = call(d, "rms", "halves")
    assert qo.shape == (2, 0, 4, 64) and rk.shape == (2, 0, 2) and not dwq.any() and not dwk.any()


@pytest.mark.parametrize("D", [128, 10])
def test_rows_of_zeros_and_extreme_values(D):
    from chunkwise_recurrent_prefill_gb300 import qk_norm_fwd
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 6, 1, D, generator=g)
    scale = torch.tensor([0.0, 1e-30, 1e-20, 1.0, 1e25, 3e37])[None, :, None, None]
    for norm, eps in (("rms", 0.0), ("l2", 0.0), ("rms", 1e-6)):
        q = (x * scale).clamp(-3e38, 3e38)
        out, _, r, _ = qk_norm_fwd(q.cuda(), q.cuda(), norm=norm, eps=eps)
        want = ref.qk(q, None, None, None, None, norm, False, eps)
        if eps == 0:
            assert out[0, 0].isnan().all() and r[0, 0].isinf().all()
        ref.close("out", out[:, 1:], want["out"][0][:, 1:], want["out"][1][:, 1:])
    out = qk_norm_fwd(torch.zeros(1, 1, 1, D, device="cuda"), torch.zeros(1, 1, 1, D, device="cuda"))[0]
    assert not out.any()


def test_what_is_not_finite_stays_in_its_head():
    d = {n: ref.gpu(v) for n, v in make(2, 20, 4, 2, 64, 64, seed=4).items()}
    clean = call(d, "rms", "halves")
    d["q"][1, 5, 2, 9] = float("nan")
    got = call(d, "rms", "halves")
    bad = torch.zeros(2, 20, 4, 64, dtype=torch.bool, device="cuda")
    bad[1, 5, 2] = True
    for i in (0, 4):
        assert torch.equal(got[i][~bad], clean[i][~bad]) and got[i][bad].isnan().all()
    for i in (1, 3, 5, 7):
        assert torch.equal(got[i], clean[i])


def test_gradient_against_differences():
    d = make(1, 7, 2, 1, 12, 8, seed=5)
    got = call({n: ref.gpu(v) for n, v in d.items()}, "rms", "pairs")
    gen = torch.Generator().manual_seed(6)
    for n, g in (("q", got[4]), ("wq", got[6])):
        base = {k: None if v is None else v.double() for k, v in d.items() if k != "positions"}
        v = torch.randn(base[n].shape, generator=gen, dtype=torch.float64)

        def loss(e):
            a = {**base, n: base[n] + e * v}
            out = ref.qk(a["q"], a["wq"], a["cos"], a["sin"], d["positions"], "rms", True, 1e-6)["out"][0]
            return (out * base["dqo"]).sum().item()

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        terms = g.cpu().double() * v
        # the difference is off by h^2 of the third derivative, the gradient by 1e-6 of its terms
        assert abs(terms.sum().item() - want) <= 2e-5 * terms.abs().sum().item() + 1e-6


@pytest.mark.parametrize("D", [64, 20])
def test_time_major_inputs(D):
    """[T, B, heads, D], and [B, heads, T, D]."""
    d = make(3, 17, 4, 2, D, D, seed=D)
    for a, b in ((0, 1), (1, 2)):
        for n in ("q", "k", "dqo", "dko"):
            d[n] = d[n].transpose(a, b).contiguous().transpose(a, b)
        check(d, "rms", "halves")


def test_more_than_32_bits_of_elements():
    from chunkwise_recurrent_prefill_gb300 import qk_norm_bwd, qk_norm_fwd
    T = (1 << 20) + 11
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.empty(1, T, 16, 136, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    k = torch.randn(1, T, 1, 136, device="cuda", generator=g).bfloat16()
    w, cut = torch.randn(136, device="cuda", generator=g), T - 1000
    c = torch.randn(T, 32, device="cuda", generator=g)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    out = qk_norm_fwd(q, k, w, w, cos=c, sin=c, positions=pos)
    last = [t[:, cut:].contiguous() for t in (q, k)]
    out2 = qk_norm_fwd(*last, w, w, cos=c, sin=c, positions=pos[:, cut:].contiguous())
    for a, b in zip(out, out2):
        assert torch.equal(a[:, cut:], b)
    rq, rk = out[2:]
    dq = qk_norm_bwd(q, k, q, k, rq, rk, w, w, cos=c, sin=c, positions=pos)[0]
    dq2 = qk_norm_bwd(*last, *last, out2[2], out2[3], w, w, cos=c, sin=c, positions=pos[:, cut:].contiguous())[0]
    assert torch.equal(dq[:, cut:], dq2)


def test_streams_and_graphs():
    from chunkwise_recurrent_prefill_gb300 import qk_norm_workspace_size
    d = {n: ref.gpu(v) for n, v in make(2, 100, 8, 2, 128, 128, "bf16", seed=9).items()}
    want = call(d, "rms", "halves")
    ws = torch.empty(qk_norm_workspace_size(d["q"], d["k"], d["cos"]), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(d, "rms", "halves")
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(d, "rms", "halves", workspace=ws)
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [
    (3, 1700, 6, 2, 128, 128),      # several rounds of a warp, a batch entry ending inside of one
    (4999, 1, 3, 5, 64, 32), (700, 7, 1, 9, 24, 16), (1, 5000, 40, 1, 8, 0),
    (2, 700, 3, 2, 384, 384), (2, 300, 3, 2, 512, 128), (2, 40, 3, 2, 320, 320)])
def test_many_tokens(B, T, Hq, Hk, D, R, io):
    check(make(B, T, Hq, Hk, D, R, io, seed=D + 1), "rms", "halves")
    check(make(B, T, Hq, Hk, D, R, io, seed=D + 2), "l2", "pairs")


@pytest.mark.parametrize("D", [64, 128])
def test_heads_side_by_side(D):
    """Queries and keys as parts of one projection's rows, heads before tokens in memory, one head of many."""
    d = make(2, 1300, 4, 2, D, D, "bf16", seed=5)
    g = torch.Generator().manual_seed(6)
    both = ref.draw(g, 2, 1300, 8 * D, io="bf16")
    d["q"], d["k"] = both[..., :4 * D].unflatten(-1, (4, D)), both[..., 5 * D:7 * D].unflatten(-1, (2, D))
    d["dqo"] = d["dqo"].transpose(1, 2).contiguous().transpose(1, 2)
    d["dko"] = ref.draw(g, 2, 1300, 9, D, io="bf16")[:, :, 3:5]
    check(d, "rms", "halves")
