"""Decay attention at the edges of its range: more heads than a grid has rows. The bounds are
those of hda_ref.py."""
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
