"""Edges of the selective state space scan."""
import pytest
import torch

import layer_ref as ref
from test_ssm_gpu import call, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("N", [16, 7])
def test_growing_segments_of_nothing(N):
    """A > 0: e^(A sum d) of a segment passes the range, but a state of zero stays zero, forward and back."""
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd
    T = 256
    d = make(2, T, 40, 1, N, "f32", seed=N, params=False, state=False)
    d["A"], d["dt"] = torch.full_like(d["A"], 3.0), torch.ones_like(d["dt"])
    late = {**d, "u": d["u"].clone()}
    late["u"][:, :T - 6] = 0
    t = {k: ref.gpu(v) for k, v in late.items()}
    o, hT = ssm_fwd(t["u"], t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], softplus=False, return_state=True, seq_splits=4)
    want = ref.scan(late, softplus=False, back=False)
    ref.close("o", o, *want["o"])
    ref.close("hT", hT, *want["hT"])
    early = {**d, "u": 0 * d["u"], "do": d["do"].clone()}
    early["do"][:, 6:] = 0
    got = call({k: ref.gpu(v) for k, v in early.items()}, softplus=False, seq_splits=4)
    want = ref.scan(early, softplus=False)
    for n, v in got.items():
        if v is not None:
            ref.close(n, v, *want[n])


def test_segments_that_grow_and_shrink():
    """A small state that grows by more than the range in a segment, and shrinks in the next: it is never large."""
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd
    T = 256
    d = make(2, T, 40, 1, 16, "f32", seed=3, params=False)
    d["A"], d["u"], d["h0"] = torch.full_like(d["A"], 0.71), 0 * d["u"], 1e-37 * d["h0"]
    d["dt"] = torch.ones_like(d["dt"])
    d["dt"][:, T // 2:] = -1
    t = {k: ref.gpu(v) for k, v in d.items()}
    o, hT = ssm_fwd(t["u"], t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], h0=t["h0"], softplus=False, return_state=True,
                    seq_splits=2)
    want = ref.scan(d, softplus=False, back=False)
    ref.close("o", o, *want["o"])
    ref.close("hT", hT, *want["hT"])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("T,C,N,splits", [(100, 40, 16, 0), (104, 40, 16, 0), (97, 64, 16, 3), (99, 7, 64, 0),
                                          (102, 33, 12, 2), (1, 5, 16, 0)])
def test_a_last_token_that_is_not_finite_leaves_dA(T, C, N, splits, value):
    """dA is made of the states before the tokens: that after the last one has no part in it."""
    t = {k: ref.gpu(v) for k, v in make(2, T, C, 1, N, "f32", seed=T).items()}
    clean = call(t, seq_splits=splits)
    t["u"][1, T - 1, 3] = value
    got = call(t, seq_splits=splits)
    assert got["o"][1, T - 1, 3].isfinite().logical_not() and got["hT"][1, 3].isfinite().logical_not().all()
    assert torch.equal(got["dA"], clean["dA"])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("N", [12, 20, 24, 36, 100])
def test_steps_of_an_infinite_input(N, io):
    """N is a multiple of 4 and no power of two: positive B and C make an infinity of an infinite u, not a NaN."""
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd, ssm_step
    g = torch.Generator().manual_seed(N)
    R, C = 3, 32
    u, dt = ref.draw(g, R, 1, C, io=io).cuda(), ref.draw(g, R, 1, C, io=io).cuda()
    b, c = (ref.draw(g, R, 1, 1, N, io=io).abs().cuda() + 1 for _ in range(2))
    A = -torch.rand(C, N, generator=g).cuda()
    u[1, 0, 5] = float("inf")
    want, h = ssm_fwd(u, dt, A, b, c, return_state=True)
    S = torch.zeros(R, C, N, device="cuda")
    o = ssm_step(u[:, 0], dt[:, 0], A, b[:, 0], c[:, 0], S)
    assert want[1, 0, 5] == float("inf") and o[1, 5] == float("inf")
    assert (S[1, 5] == float("inf")).all() and (h[1, 5] == float("inf")).all()
    o[1, 5] = want[1, 0, 5] = 0
    assert o.isfinite().all() and want.isfinite().all()


@pytest.mark.parametrize("lo,hi", [(-80.0, -20.0), (-20.0, -5.0), (-5.0, 0.0), (0.0, 20.0)])
def test_small_steps_keep_their_digits(lo, hi):
    """Step sizes on their own: with A = 0, u = B = C = do = 1 the state after one token, and du, are the step. Whatever
    the size of x, softplus(x) is off by the hardware's 2^x (2^-22 of the value, four U), by a rounding each of what the
    argument's rounding left out, of the last two sums and of the polynomial's terms before (less than one U
    together), and by its fit (a tenth of a U): eight U. (What the argument's rounding leaves out has an error of its own
    of 2^-24 of 2^-19.)"""
    from chunkwise_recurrent_prefill_gb300 import ssm_bwd, ssm_fwd, ssm_step
    C = 4096
    x = torch.linspace(lo, hi, C)
    want = torch.logaddexp(x.double(), torch.zeros(C).double())
    dt, one, A, b = x.cuda()[None, None], torch.ones(1, 1, C, device="cuda"), torch.zeros(C, 1, device="cuda"), \
        torch.ones(1, 1, 1, 1, device="cuda")
    hT = ssm_fwd(one, dt, A, b, b, return_state=True)[1]
    S = torch.zeros(1, C, 1, device="cuda")
    ssm_step(one[:, 0], dt[:, 0], A, b[:, 0], b[:, 0], S)
    du = ssm_bwd(one, one, dt, A, b, b)[0]
    for n, got in (("hT", hT), ("S", S), ("du", du)):
        ref.close(n, got.view(C), want, 8 * ref.U * want)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("off", [-float("inf"), torch.finfo(torch.bfloat16).min, -1e30])
def test_tokens_that_a_mask_takes_out(off, io):
    """dt of minus infinity, or the type's lowest value: steps of zero, which leave the state and have no gradient."""
    from chunkwise_recurrent_prefill_gb300 import ssm_step
    d = make(2, 29, 40, 1, 16, io, seed=2)
    d["dt"][:, 5:] = off
    t = {k: ref.gpu(v) for k, v in d.items()}
    got = call(t)
    want = ref.scan({**{k: v if k in ("A", "D", "dt_bias", "h0") else v[:, :5] for k, v in d.items() if k != "dhT"}}, io=io,
                    back=False)
    ref.close("hT", got["hT"], *want["hT"])
    S = got["hT"].clone()
    o = ssm_step(t["u"][:, 9], t["dt"][:, 9], t["A"], t["Bm"][:, 9], t["Cm"][:, 9], S, D=t["D"], z=t["z"][:, 9],
                 dt_bias=t["dt_bias"])
    assert torch.equal(S, got["hT"]) and not got["ddt"][:, 5:].any() and not got["dB"][:, 5:].any()
    # (sums of N products in another order, of values below 100)
    assert torch.allclose(o.float(), got["o"][:, 9].float(), rtol=2.0 ** -7 if io == "bf16" else 1e-5, atol=1e-4)
    for n, v in got.items():
        assert v.isfinite().all(), n


def test_steps_that_are_not_finite():
    """softplus of an infinity is one, and that of a NaN a NaN."""
    from chunkwise_recurrent_prefill_gb300 import ssm_fwd, ssm_step
    for io in ("bf16", "f32"):
        T = torch.bfloat16 if io == "bf16" else torch.float32
        one = torch.ones(1, 1, 3, device="cuda", dtype=T)
        dt = torch.tensor([[[float("inf"), float("nan"), 3e38]]], device="cuda").to(T)
        A, b = torch.zeros(3, 1, device="cuda"), torch.ones(1, 1, 1, 1, device="cuda", dtype=T)
        A[0] = -1
        S = torch.zeros(1, 3, 1, device="cuda")
        ssm_step(one[:, 0], dt[:, 0], A, b[:, 0], b[:, 0], S)
        for h in (ssm_fwd(one, dt, A, b, b, return_state=True)[1], S):
            assert h[0, 0] == float("inf") and h[0, 1].isnan() and h[0, 2] == dt[0, 0, 2].float()


def test_gradients_of_more_than_32_bits_of_elements():
    """The last tokens' gradients, of inputs past 2^31 elements, against those of the same tokens on their own."""
    from chunkwise_recurrent_prefill_gb300 import last_device_status, ssm_bwd, ssm_fwd
    T, C, N = (1 << 20) + 11, 2080, 8
    g = torch.Generator("cuda").manual_seed(2)
    u, dt, z, do = (torch.empty(1, T, C, device="cuda", dtype=torch.bfloat16).normal_(generator=g) for _ in range(4))
    Bm, Cm = (torch.randn(1, T, 1, N, device="cuda", generator=g).bfloat16() for _ in range(2))
    A = -torch.rand(C, N, device="cuda", generator=g) - 0.5
    cut = T - 1000
    du, ddt, _, dBm, dCm, _, dz, _, _ = ssm_bwd(do, u, dt, A, Bm, Cm, z=z)
    whole = [x[:, cut:].clone() for x in (du, ddt, dBm, dCm, dz)]
    del du, ddt, dz
    head = [x[:, :cut] for x in (u, dt)] + [A] + [x[:, :cut] for x in (Bm, Cm)]
    h = ssm_fwd(*head, return_state=True)[1]
    part = [x[:, cut:].contiguous() for x in (u, dt)] + [A] + [x[:, cut:].contiguous() for x in (Bm, Cm)]
    own = ssm_bwd(do[:, cut:].contiguous(), *part, z=z[:, cut:].contiguous(), h0=h)
    assert last_device_status() == 0
    # the same operations but for where a chunk ends, each rounded to bf16
    for n, a, b in zip(("du", "ddt", "dB", "dC", "dz"), whole, (own[0], own[1], own[3], own[4], own[6])):
        a, b = a.float(), b.float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-3 * b.square().mean().sqrt()).all(), n
