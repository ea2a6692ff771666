"""Decay attention at the edges of its range: infinite values, and more heads than a grid
has rows. The bounds are those of hda_ref.py."""
import pytest
import torch

import hda_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _gpu(x):
    return {n: ref.to_gpu(t) for n, t in x.items()}


def _abs(a, keep):
    return [t.abs() if isinstance(t, torch.Tensor) and i != keep else t for i, t in enumerate(a)]


def same_pattern(name, got, want, absolute, size, T, D):
    """NaN where the 64-bit form has NaN, the same infinities, finite values within their bounds; not
    where the growth of the state alone (size: the sum of absolute values without the infinite ones)
    comes near the largest float, which the 64-bit form does not know of."""
    near = size > 2.0 ** 100
    got64, want = got.cpu().double().masked_fill(near, 0.0), want.masked_fill(near, 0.0)
    assert torch.equal(got64.isnan(), want.isnan()), f"{name}: NaN elsewhere"
    inf = want.isinf()
    assert torch.equal(got64.isinf(), inf) and torch.equal(got64[inf], want[inf]), f"{name}: infinities"
    fine = want.isfinite() & ~near
    ref.check(name, got64[fine].float(), want[fine], absolute[fine], T, D)


def _finite(a, keep):
    return [t.abs().nan_to_num(posinf=1.0) if isinstance(t, torch.Tensor) and i != keep else t
            for i, t in enumerate(a)]


# ---------------------------------------------------------------- infinite values
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("T", [1, 16, 77, 150])
@pytest.mark.parametrize("decay", [0.0, -1e-6, -0.02, -0.6, -3.0, 0.01, 0.6])
def test_infinite_values_are_those_of_the_recurrence(decay, T, splits):
    """An infinite k, v or do makes an infinite state, which a decay leaves infinite, through the
    tokens after it and a last tile that is not full."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd
    x = ref.inputs(1, T, 2, 2, 2, 2, 24, 40, io="f32", seed=T, decay=[decay, decay])
    x["k"][0, T // 10, 0, 3] = float("inf")
    x["v"][0, T // 4, 1, 5] = float("-inf")
    x["do"][0, T // 2, 0, 7] = float("inf")
    g = _gpu(x)
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"])
    got = hda_fwd(g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], return_state=True,
                  path="exact", seq_splits=splits)
    for n, o, w, b, z in zip(("o", "hT"), got, ref.forward(*a), ref.forward(*_abs(a, 3)),
                             ref.forward(*_finite(a, 3))):
        same_pattern(n, o, w, b, z, T, 40)
    got = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], g["dhT"],
                  path="exact", seq_splits=splits)
    a = (x["do"],) + a + (x["dhT"],)
    for n, o, w, b, z in zip(("dq", "dk", "dv", "dh0"), got, ref.backward(*a), ref.backward(*_abs(a, 4)),
                             ref.backward(*_finite(a, 4))):
        same_pattern(n, o, w, b, z, T, 40)


# ---------------------------------------------------------------- many heads
@pytest.mark.parametrize("B,H,T", [(1, 70000, 3), (2, 40000, 2), (1, 65537, 20)])
def test_more_heads_than_a_grid_has_rows(B, H, T):
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd, last_device_status
    x = ref.inputs(B, T, H, H, 1, H, 8, 8, io="f32", seed=H)
    x["decay"] = -2.0 ** -torch.linspace(-2.0, 8.0, H)
    g = _gpu(x)
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"])
    got = hda_fwd(g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], return_state=True)
    for n, o, w, b in zip(("o", "hT"), got, ref.forward(*a), ref.forward(*_abs(a, 3))):
        ref.check(n, o, w, b, T, 8)
    got = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], g["dhT"])
    a = (x["do"],) + a + (x["dhT"],)
    want, absolute = ref.backward(*a), ref.backward(*_abs(a, 4))
    for i, n in ((0, "dq"), (2, "dv"), (3, "dh0")):
        ref.check(n, got[i], want[i], absolute[i], T, 8)
    # the gradient of the one k head is a sum over H more terms, each addition rounding once
    err = (got[1].cpu().double() - want[1]).abs()
    assert (err <= (ref.roundings(T, 8) + H) * ref.U * absolute[1]).all()
    assert last_device_status() == 0
