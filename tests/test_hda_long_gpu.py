"""Sequences of many chunks on the tensor cores: the steady state of a split sequence, and the accuracy
of returned states. The bounds are derived in hda_ref.py, and at the test; the 64-bit form runs on the
GPU."""
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


def _on_gpu(a):
    return [t.cuda() if isinstance(t, torch.Tensor) else t for t in a]


# B, T, H, Hq, Hk, Hv, Dk, Dv; splits. On 152 SMs: chunks of a state CTA and its pieces
LONG = [
    ((1, 64 * 41 + 5, 40, 40, 10, 40, 64, 64), 2),     # 20 and 21 chunks, one piece
    ((2, 64 * 41 + 5, 12, 12, 12, 3, 128, 64), 2),     # 7, three pieces of a segment
    ((1, 64 * 45, 2, 2, 1, 2, 128, 128), 2),           # 4 or 5, five pieces
    ((1, 64 * 60 + 1, 2, 2, 2, 2, 64, 128), 20),       # 20 start states: two batches of the scan
    ((1, 64 * 150 + 33, 20, 20, 20, 20, 64, 64), 3),   # 25, two pieces
]


@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("shape,splits", LONG)
def test_split_sequences_of_many_chunks(shape, splits, state):
    """The state pass with more chunks to a CTA than it has stages and accumulators, several pieces
    to a segment, and more pieces than a batch of the scan; with the final state (three parts of its
    operand) and without (two)."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd, last_device_status
    x = ref.inputs(*shape, io="bf16", seed=splits, strided=True)
    x["decay"] = -2.0 ** -torch.linspace(1.0, 11.0, shape[2])
    g = _gpu(x)
    T, Dk, Dv = shape[1], shape[6], shape[7]
    a = _on_gpu((x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"]))
    o, hT = hda_fwd(g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], return_state=state,
                    path="tc", seq_splits=splits)
    want, absolute = ref.forward(*a), ref.forward(*_abs(a, 3))
    ref.check("o", o, want[0].cpu(), absolute[0].cpu(), T, Dk, "tc")
    if state:
        ref.check("hT", hT, want[1].cpu(), absolute[1].cpu(), T, Dk, "tc", state=True)
    # with no initial state given there is no dh0
    h0 = x["h0"] if state else torch.zeros_like(x["h0"])
    a = _on_gpu((x["do"], x["q"], x["k"], x["v"], x["decay"], x["scale"], h0, x["dhT"]))
    got = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"] if state else None,
                  g["dhT"], path="tc", seq_splits=splits)
    want, absolute = ref.backward(*a), ref.backward(*_abs(a, 4))
    for n, d, w, b in zip(("dq", "dk", "dv"), got, want, absolute):
        ref.check(n, d, w.cpu(), b.cpu(), T, max(Dk, Dv), "tc")
    if state:
        ref.check("dh0", got[3], want[3].cpu(), absolute[3].cpu(), T, max(Dk, Dv), "tc", state=True)
    assert last_device_status() == 0


@pytest.mark.parametrize("shape,splits", [((1, 64 * 40 + 5, 8, 8, 8, 8, 128, 128), 1), LONG[0], LONG[4]])
def test_returned_states_keep_fp32_accuracy(shape, splits):
    """hT and dh0 to 2^-20 = 1e-6 of their root mean square. Three parts of the operand hold all 24
    bits of a term; what is left are the decay's two roundings (2^-24 each) and the tensor core's sums,
    which cut 2^-24 on the average at each step: 24 steps of an accumulator of two chunks, all but the
    last few on a part of the sum. Two parts would cut 2^-17 of each
    term on the average, always towards zero: 8e-6 of the sum."""
    from chunkwise_recurrent_prefill_gb300 import hda_bwd, hda_fwd
    x = ref.inputs(*shape, io="bf16", seed=splits + 50)
    x["decay"] = -2.0 ** -torch.linspace(7.0, 11.0, shape[2])
    g = _gpu(x)
    a = _on_gpu((x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"]))
    _, hT = hda_fwd(g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], return_state=True,
                    path="tc", seq_splits=splits)
    dh0 = hda_bwd(g["do"], g["q"], g["k"], g["v"], g["decay"], x["scale"], g["h0"], g["dhT"],
                  path="tc", seq_splits=splits)[3]
    a = _on_gpu((x["do"], x["q"], x["k"], x["v"], x["decay"], x["scale"], x["h0"], x["dhT"]))
    for n, s, w in (("hT", hT, ref.forward(*a[1:7])[1]), ("dh0", dh0, ref.backward(*a)[3])):
        rms = ((s.double() - w).square().mean() / w.square().mean()).sqrt().item()
        assert rms <= 2.0 ** -20, f"{n}: rms error {rms:.3g} of the state's"
