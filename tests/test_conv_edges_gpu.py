"""The short convolution where vectors of channels end and start: rows on 8 bytes but not on 16, and on none of them."""
import pytest
import torch

import layer_ref as ref
from test_conv_gpu import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("C", [4, 12, 44, 132, 46])
@pytest.mark.parametrize("lo,wide", [(0, 0), (4, 4), (4, 0), (2, 2), (8, 4), (0, 12)])
def test_alignment(lo, wide, C, io):
    """x and dy from element ``lo`` of rows that are ``wide`` longer: both, and each of them beside a contiguous one."""
    from chunkwise_recurrent_prefill_gb300 import conv_bwd, conv_fwd, last_device_status
    d = make(3, 41, C, 4, io, seed=C + lo)
    cut = {}
    t = {n: ref.gpu(v) for n, v in d.items()}
    for n in ("x", "dy"):
        rows = torch.zeros(3, 41, lo + C + wide, dtype=d[n].dtype, device="cuda")
        cut[n] = rows[..., lo:lo + C].copy_(t[n])
    want = ref.conv(d["x"], d["w"], d["bias"], d["s0"], d["dy"], d["dsT"], "silu", io)
    for names in (("x", "dy"), ("x",), ("dy",)):
        a = {**t, **{n: cut[n] for n in names}}
        y, sT = conv_fwd(a["x"], a["w"], a["bias"], a["s0"], act="silu", return_state=True)
        grads = conv_bwd(a["dy"], a["x"], a["w"], a["bias"], a["s0"], a["dsT"], act="silu")
        for n, v in zip(("y", "sT", "dx", "dw", "db", "ds0"), (y, sT) + grads):
            ref.close(n, v, *want[n])
    assert last_device_status() == 0

