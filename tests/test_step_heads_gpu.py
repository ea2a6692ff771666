"""hda_step with more heads than a product of two head counts in 32 bits allows (the bounds are
derived in hda_ref.py)."""
import pytest
import torch

import hda_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("H,Hq,Hk", [(65536, 65536, 65536), (46400, 46400, 23200), (98304, 1, 49152)])
def test_step_of_many_heads(H, Hq, Hk):
    from chunkwise_recurrent_prefill_gb300 import hda_step, last_device_status
    x = ref.inputs(2, 1, H, Hq, Hk, H, 2, 4, "f32", seed=H % 97)
    x["decay"] = -2.0 ** -torch.linspace(-2.0, 8.0, H)
    q, k, v, decay, S = (x[n].cuda() for n in ("q", "k", "v", "decay", "h0"))
    o = hda_step(q[:, 0], k[:, 0], v[:, 0], decay, x["scale"], S)
    assert last_device_status() == 0
    a = (x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"])
    want = ref.forward(*a)
    absolute = ref.forward(*[t.abs() if isinstance(t, torch.Tensor) and i != 3 else t for i, t in enumerate(a)])
    ref.check("o", o[:, None], want[0], absolute[0], 1, 2)
    ref.check("S", S, want[1], absolute[1], 1, 2, state=True)
