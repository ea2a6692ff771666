"""What the bindings of the short convolution, the selective scan and the norm of queries and keys refuse (CPU
tensors: nothing is launched)."""
import numpy as np
import pytest
import torch

import chunkwise_recurrent_prefill_gb300 as pkg
from chunkwise_recurrent_prefill_gb300 import build_ext, conv, qk_norm, ssm


@pytest.fixture(autouse=True)
def launched(monkeypatch):
    """CPU stands for the device; launches are noted."""
    build_ext.build()
    calls = []
    params = conv._params

    def on_device(x, w, bias):
        s = Seems(x)
        s.shape = x.shape
        return params(s, w, bias).d

    monkeypatch.setattr(conv, "_params", on_device)
    for mod in (conv, ssm, qk_norm):
        monkeypatch.setattr(mod, "_launch", lambda *a: calls.append(a) or 0)
    inputs = ssm._check_inputs
    monkeypatch.setattr(ssm, "_check_inputs", lambda sh, u, *a: inputs(sh, Seems(u), *a).d)
    heads = qk_norm._check_inputs
    monkeypatch.setattr(qk_norm, "_check_inputs", lambda sh, q, *a: heads(sh, Seems(q), *a).d)
    return calls


class Seems:
    """A tensor whose device says that it is a GPU, and equals the CPU."""

    class Device:
        type = "cuda"

        def __init__(self, d):
            self.d = d

        def __eq__(self, other):
            return self.d == other

        def __ne__(self, other):
            return self.d != other

        __hash__ = None

    def __init__(self, t):
        self.device = self.Device(t.device)


def test_a_host_tensor_is_refused(monkeypatch):
    monkeypatch.undo()
    x, w = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.conv_fwd(x, w)
    b = torch.zeros(1, 4, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.ssm_fwd(x, x, torch.zeros(8, 16), b, b)
    q = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.qk_norm_fwd(q, q)


def test_conv():
    x, w, S = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(3, 3, 8)
    for bad in (None, [0.0], np.zeros((8, 4), np.float32)):
        with pytest.raises(TypeError, match="w must be"):
            pkg.conv_fwd(x, bad)
        with pytest.raises(TypeError, match="dy must be"):
            pkg.conv_bwd(bad, x, w)
        with pytest.raises(TypeError, match="S must be"):
            pkg.conv_step(x[:, 0], w, bad)
    for args, kw, what in (((x.half(), w), {}, "bfloat16"), ((x, w.double()), {}, "dtype"), ((x, w, w[:, 0].bfloat16()), {}, "dtype")):
        with pytest.raises(TypeError, match=what):
            pkg.conv_fwd(*args, **kw)
    for args, kw, what in (((x[0], w), {}, "B, T, C"), ((x, w[0]), {}, "C, W"), ((x, w[:4]), {}, "shape"),
                           ((x, w), dict(act="relu"), "act"), ((x.transpose(1, 2), w[:5].contiguous()), {}, "contiguous"),
                           ((x.expand(2, 5, 8)[:, :1].expand(2, 5, 8), w), {}, "strides"),
                           ((x, w, None, torch.zeros(2, 4, 8)), {}, "s0: shape"),
                           ((x, w), dict(sT=torch.zeros(2, 3, 7)), "sT: shape"), ((x, w), dict(y=torch.zeros(2, 5, 4)), "y: shape")):
        with pytest.raises(ValueError, match=what):
            pkg.conv_fwd(*args, **kw)
    with pytest.raises(ValueError, match="dy: shape"):
        pkg.conv_bwd(x[:, :4], x, w)
    with pytest.raises(TypeError, match="slots: dtype"):
        pkg.conv_step(x[:, 0], w, S, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="S: shape"):
        pkg.conv_step(x[:, 0], w, S[:, :2].contiguous())


def test_scan(launched):
    u, A, b = torch.zeros(2, 5, 8), torch.zeros(8, 16), torch.zeros(2, 5, 2, 16)
    for bad in (None, [0.0], np.zeros((8, 16), np.float32)):
        with pytest.raises(TypeError, match="A must be"):
            pkg.ssm_fwd(u, u, bad, b, b)
        with pytest.raises(TypeError, match="dt must be"):
            pkg.ssm_fwd(u, bad, A, b, b)
        with pytest.raises(TypeError, match="do must be"):
            pkg.ssm_bwd(bad, u, u, A, b, b)
        with pytest.raises(TypeError, match="S must be"):
            pkg.ssm_step(u[:, 0], u[:, 0], A, b[:, 0], b[:, 0], bad)
    with pytest.raises(TypeError, match="bfloat16"):
        pkg.ssm_fwd(u.double(), u, A, b, b)
    for args, kw, err, what in (
            ((u, u.bfloat16(), A, b, b), {}, TypeError, "dt: dtype"), ((u, u, A, b, b), dict(z=u.bfloat16()), TypeError, "z: dtype"),
            ((u, u, A.bfloat16(), b, b), {}, TypeError, "A: dtype"), ((u[0], u, A, b, b), {}, ValueError, "B, T, C"),
            ((u, u, A[0], b, b), {}, ValueError, "C, N"), ((u, u, A, b[:, :, 0], b), {}, ValueError, "B, T, G, N"),
            ((u, u, A, b, b[:, :, :1]), {}, ValueError, "Cm: shape"), ((u, u, A, b[..., :8], b), {}, ValueError, "Bm: shape"),
            ((u, u, A, torch.zeros(2, 5, 2, 32)[..., :16], b), {}, ValueError, "groups"),
            ((u, u, A, b, b), dict(D=torch.zeros(7)), ValueError, "D: shape"),
            ((u, u, A, b, b), dict(h0=torch.zeros(2, 8, 8)), ValueError, "h0: shape"),
            ((u, u, A, b, b), dict(hT=torch.zeros(1, 8, 16)), ValueError, "hT: shape"),
            ((u, u, A, b, b), dict(o=torch.zeros(2, 5, 9)), ValueError, "o: shape")):
        with pytest.raises(err, match=what):
            pkg.ssm_fwd(*args, **kw)
    assert not launched
    pkg.ssm_fwd(u, u, A, b, b)
    assert len(launched) == 1


def test_qk(launched):
    q, k, w = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 2, 16), torch.ones(16)
    c = torch.zeros(9, 8)
    for bad in (None, [0.0], np.zeros(16, np.float32)):
        with pytest.raises(TypeError, match="k must be"):
            pkg.qk_norm_fwd(q, bad)
        with pytest.raises(TypeError, match="dko must be"):
            pkg.qk_norm_bwd(q, bad, q, k, None, None)
    with pytest.raises(TypeError, match="rq must be"):
        pkg.qk_norm_bwd(q, k, q, k, None, None)
    for args, kw, err, what in (
            ((q.half(), k), {}, TypeError, "bfloat16"), ((q, k.bfloat16()), {}, TypeError, "k: dtype"),
            ((q[0], k), {}, ValueError, "heads"), ((q, k[..., :8]), {}, ValueError, "k: shape"), ((q, k[:1]), {}, ValueError, "k: shape"),
            ((q, k), dict(norm="layer"), ValueError, "norm"), ((q, k), dict(layout="thirds"), ValueError, "layout"),
            ((q, k, w[:8]), {}, ValueError, "wq: shape"), ((q, k), dict(cos=c), ValueError, "go together"),
            ((q, k), dict(cos=c, sin=c[:8]), ValueError, "sin: shape"), ((q, k), dict(cos=c[0], sin=c[0]), ValueError, "cos must be"),
            ((q, k), dict(positions=torch.zeros(2, 5)), TypeError, "positions: dtype"),
            ((q, k), dict(positions=torch.zeros(5, dtype=torch.int32)), ValueError, "positions: shape"),
            ((q, k), dict(qo=torch.zeros(2, 5, 4, 8)), ValueError, "qo: shape")):
        with pytest.raises(err, match=what):
            pkg.qk_norm_fwd(*args, **kw)
    assert not launched
    assert pkg.qk_norm_fwd(q, k, norm="none")[2:] == (None, None) and len(launched) == 1


def test_workspaces_elsewhere(launched):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    A, b = torch.zeros(8, 16), torch.zeros(2, 5, 2, 16)
    q, r = torch.zeros(2, 5, 4, 16), torch.zeros(2, 5, 4)
    for call in (lambda ws: pkg.conv_bwd(x, x, w, workspace=ws), lambda ws: pkg.ssm_fwd(x, x, A, b, b, workspace=ws),
                 lambda ws: pkg.ssm_bwd(x, x, x, A, b, b, workspace=ws),
                 lambda ws: pkg.qk_norm_bwd(q, q, q, q, r, r, workspace=ws)):
        n = len(launched)
        for bad in (torch.empty(64, device="meta"), torch.zeros(64)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(bad)
        with pytest.raises(TypeError, match="workspace"):
            call(1 << 20)
        assert len(launched) == n
        call(torch.zeros(64))
        assert len(launched) == n + 1
