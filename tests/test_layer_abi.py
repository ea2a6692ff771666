"""Argument checks of the short convolution, the selective scan and the norm of queries and keys on fake device
addresses: every call here is refused on the host (or has nothing to launch). Run where no GPU is visible."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only checks on fake device addresses: run where no GPU is visible")
    from chunkwise_recurrent_prefill_gb300 import build_ext
    from chunkwise_recurrent_prefill_gb300.gla import load_library
    build_ext.build()
    return load_library()


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def at(i):
    return None if i is None else i << 36


def fill(sh, **kw):
    for n, v in kw.items():
        if isinstance(v, tuple):
            for f, x in zip(getattr(sh, n)._fields_, v):
                setattr(getattr(sh, n), f[0], x)
        else:
            setattr(sh, n, v)
    return sh


def test_exports(lib):
    src = open(os.path.join(ROOT, "include", "gla.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b((?:ssm|gla_conv|gla_qk_norm)_[a-z0-9_]+)\s*\(", src))
    assert {"ssm_fwd", "ssm_bwd", "ssm_step", "gla_conv_fwd", "gla_conv_bwd", "gla_conv_step", "gla_qk_norm_fwd",
            "gla_qk_norm_bwd", "ssm_fwd_workspace_size", "ssm_bwd_workspace_size", "gla_conv_bwd_workspace_size",
            "gla_qk_norm_bwd_workspace_size"} == names
    assert all(hasattr(lib, n) for n in names)


class Call:
    """A C entry with pointers i << 36 (None: NULL); call(i, value) replaces one, keywords change the shape."""

    def __init__(self, f, pointers, shape, tail):
        self.f, self.pointers, self.shape, self.tail = f, pointers, shape, tail

    def __call__(self, i=None, value=None, **kw):
        p = [at(x) for x in self.pointers]
        if i is not None:
            p[i] = value
        tail = {k: kw.pop(k, v) for k, v in self.tail.items()}
        P = [tail.pop("P")] if "P" in tail else []
        sh = fill(self.shape(), **kw)
        return self.f(*(vp(x) for x in p), *P, ctypes.byref(sh), *tail.values(), None)


def conv_shape():
    from chunkwise_recurrent_prefill_gb300.gla import _ConvShape
    return _ConvShape(B=2, T=10, C=64, W=4, act=1, io=0)


def test_conv_checks(lib):
    from chunkwise_recurrent_prefill_gb300.gla import _ConvShape
    fwd = Call(lib.gla_conv_fwd, [1, 2, None, 4, 5, 6], conv_shape, {})      # x w bias s0 y sT
    assert fwd() in (6, 8)                                  # all in order: no device to run on
    for i in (0, 1, 4):
        assert fwd(i, None) == 1
    assert lib.gla_conv_fwd(*[None] * 6, ctypes.POINTER(_ConvShape)(), None) == 1
    assert fwd(B=-1) == 2 and fwd(T=-1) == 2 and fwd(C=-8) == 2 and fwd(C=(1 << 20) + 1) == 2
    assert fwd(B=1 << 30, T=1 << 30) == 2 and fwd(B=1 << 20, T=1 << 10, C=1 << 20) == 2
    assert fwd(W=0) == 3 and fwd(W=9) == 3
    assert fwd(0, at(1) + 1) == 4 and fwd(4, at(5) + 8) == 4 and fwd(3, at(4) + 2) == 4 and fwd(1, at(2) + 2) == 4
    assert fwd(0, at(1) + 2) in (6, 8)                      # x only needs its element's alignment
    assert fwd(4, at(1) + 1024) == 5 and fwd(5, at(5)) == 5 and fwd(4, at(2)) == 5
    assert fwd(io=2) == 10 and fwd(act=3) == 10 and fwd(act=-1) == 10
    # strides
    assert fwd(x=(10 * 128, 128)) in (6, 8) and fwd(x=(10 * 128, -128)) == 2 and fwd(x=(0, 128)) == 2
    assert fwd(x=(1 << 61, 128)) == 2
    assert fwd(B=1, x=(-7, 128)) in (6, 8)                  # a dimension of one element may say anything
    assert fwd(4, at(1) + 4096, B=1, x=(0, 1 << 20)) == 5   # y laid inside the gaps of a strided x
    bwd = Call(lib.gla_conv_bwd, [1, 2, 3, None, 5, 6, 7, 8, None, 10], conv_shape, dict(ws=None, n=0))
    assert bwd() in (6, 8)                                  # dy x w bias s0 dsT dx dw dbias ds0
    for i in (0, 1, 2, 6):
        assert bwd(i, None) == 1
    assert bwd(7, at(3)) == 5 and bwd(9, at(5)) == 5 and bwd(6, at(1)) == 5 and bwd(7, at(7)) == 5
    assert bwd(dy=(5, 0)) == 2 and bwd(6, at(7) + 4) == 4
    step = Call(lib.gla_conv_step, [1, 2, None, 4, 5, 6], conv_shape, dict(P=4))     # x w bias S slots y
    assert step() in (6, 8) and step(T=-5, x=(64, -3)) in (6, 8)     # T and x.t are not looked at
    assert step(0, None) == 1 and step(3, None) == 1 and step(5, None) == 1 and step(3, None, W=1) in (6, 8)
    assert step(P=-1) == 2 and step(4, None, P=1) == 2
    assert step(4, at(5) + 2) == 4 and step(3, at(4) + 8) == 4 and step(5, at(4)) == 5 and step(3, at(1)) == 5


def ssm_shape():
    from chunkwise_recurrent_prefill_gb300.gla import _SsmShape
    return _SsmShape(B=2, T=10, C=64, G=2, N=16, softplus=1, io=0)


def test_scan_checks(lib):
    from chunkwise_recurrent_prefill_gb300.gla import _Options, _SsmShape, options
    opt = ctypes.POINTER(_Options)()
    # u dt A B C D z dt_bias h0 o hT
    fwd = Call(lib.ssm_fwd, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], ssm_shape, dict(opt=opt))
    assert fwd() in (6, 8)
    for i in (0, 1, 2, 3, 4, 9):
        assert fwd(i, None) == 1
    for i in (5, 6, 7, 8, 10):
        assert fwd(i, None) in (6, 8)
    assert lib.ssm_fwd(*[None] * 11, ctypes.POINTER(_SsmShape)(), None, None) == 1
    assert fwd(B=-1) == 2 and fwd(T=-1) == 2 and fwd(G=3) == 2 and fwd(G=0) == 2 and fwd(C=-64) == 2
    assert fwd(B=1 << 26, C=1 << 10) == 2 and fwd(T=1 << 31) == 2 and fwd(B=1 << 15, T=1 << 15, G=64, N=128) == 2
    assert fwd(N=0) == 3 and fwd(N=129) == 3
    assert fwd(0, at(1) + 1) == 4 and fwd(2, at(3) + 2) == 4 and fwd(8, at(9) + 4) == 4 and fwd(9, at(10) + 8) == 4
    assert fwd(3, at(4) + 2) in (6, 8)
    assert fwd(9, at(7)) == 5 and fwd(10, at(9)) == 5 and fwd(10, at(10)) == 5 and fwd(9, at(3) + 64) == 5
    assert fwd(io=2) == 10 and fwd(softplus=2) == 10
    assert fwd(opt=ctypes.byref(options("tc"))) == 10 and fwd(opt=ctypes.byref(options("auto", -1))) == 10
    assert fwd(opt=ctypes.byref(options("auto", 0, None, "scalar"))) == 10
    assert fwd(b=(10 * 40, 40)) in (6, 8) and fwd(b=(10 * 40, 0)) == 2 and fwd(z=(640, -64)) == 2
    # do u dt A B C D z dt_bias h0 dhT | du ddt dA dB dC dD dz ddt_bias dh0
    bwd = Call(lib.ssm_bwd, list(range(1, 21)), ssm_shape, dict(opt=opt))
    assert bwd() in (6, 8)
    for i in (0, 1, 2, 3, 4, 5, 11, 12, 13, 14, 15):
        assert bwd(i, None) == 1
    for i in (6, 8, 9, 10, 16, 17, 18, 19):
        assert bwd(i, None) in (6, 8)
    assert bwd(7, None) == 1                                # dz without z
    assert bwd(11, at(12) + 8) == 4 and bwd(14, at(15) + 2) == 4 and bwd(16, at(17) + 1) == 4
    assert bwd(19, at(10)) == 5 and bwd(15, at(15)) == 5 and bwd(13, at(4)) == 5 and bwd(17, at(8)) == 5
    # u dt A B C D z dt_bias S slots o
    step = Call(lib.ssm_step, [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11], ssm_shape, dict(P=4))
    assert step() in (6, 8) and step(T=-1, u=(64, -3)) in (6, 8)
    for i in (0, 2, 4, 8, 10):
        assert step(i, None) == 1
    assert step(P=-1) == 2 and step(9, None, P=1) == 2 and step(9, None, P=2) in (6, 8)
    assert step(8, at(9) + 4) == 4 and step(9, at(10) + 2) == 4 and step(10, at(9)) == 5 and step(8, at(3)) == 5


def test_scan_workspaces(lib):
    from chunkwise_recurrent_prefill_gb300.gla import options
    def size(f, splits=0, **kw):
        return f(ctypes.byref(fill(ssm_shape(), **kw)), ctypes.byref(options("auto", splits)))
    assert size(lib.ssm_fwd_workspace_size) > 0 and size(lib.ssm_fwd_workspace_size, N=0) == 0
    assert size(lib.ssm_fwd_workspace_size, T=0) == 0 and size(lib.ssm_fwd_workspace_size, -1) == 0
    # segments' states
    a, b = (size(lib.ssm_fwd_workspace_size, n, T=800) for n in (1, 10))
    assert b - a >= 2 * 10 * 64 * 16 * 4
    # more segments than chunks of tokens are as many as those
    assert size(lib.ssm_fwd_workspace_size, 1000, T=80) == size(lib.ssm_fwd_workspace_size, 10, T=80)
    assert size(lib.ssm_bwd_workspace_size, T=800) > size(lib.ssm_fwd_workspace_size, T=800)


def qk_shape():
    from chunkwise_recurrent_prefill_gb300.gla import _QkShape
    return _QkShape(B=2, T=10, Hq=4, Hk=2, D=64, R=64, P=100, eps=1e-6, norm=1, pairs=0, io=0)


def test_qk_checks(lib):
    from chunkwise_recurrent_prefill_gb300.gla import _QkShape
    # q k wq wk cos sin positions | qo ko rq rk
    fwd = Call(lib.gla_qk_norm_fwd, list(range(1, 12)), qk_shape, {})
    assert fwd() in (6, 8)
    for i in (0, 1, 4, 5, 7, 8):
        assert fwd(i, None) == 1
    for i in (2, 3, 6, 9, 10):
        assert fwd(i, None) in (6, 8)
    assert fwd(4, None, R=0) in (6, 8) and fwd(1, None, Hk=0) in (6, 8)
    assert lib.gla_qk_norm_fwd(*[None] * 11, ctypes.POINTER(_QkShape)(), None) == 1
    assert fwd(B=-1) == 2 and fwd(Hq=-1) == 2 and fwd(R=63) == 2 and fwd(R=66) == 2 and fwd(P=-1) == 2
    assert fwd(P=1 << 31) == 2 and fwd(B=1 << 30, T=1 << 30) == 2
    assert fwd(D=0, R=0) == 3 and fwd(D=1025) == 3
    assert fwd(0, at(1) + 1) == 4 and fwd(7, at(8) + 8) == 4 and fwd(4, at(5) + 2) == 4 and fwd(6, at(7) + 2) == 4
    assert fwd(7, at(1)) == 5 and fwd(8, at(8)) == 5 and fwd(9, at(8) + 64) == 5 and fwd(10, at(7)) == 5
    assert fwd(norm=3) == 10 and fwd(pairs=2) == 10 and fwd(io=5) == 10
    assert fwd(eps=-1.0) == 10 and fwd(eps=float("nan")) == 10
    assert fwd(norm=0) == 10                                # weights without a norm
    assert fwd(q=(0, 256, 64)) == 2 and fwd(q=(2560, 256, -64)) == 2 and fwd(k=(2560, 256, 65)) in (6, 8)
    # dqo dko q k rq rk wq wk cos sin positions | dq dk dwq dwk
    bwd = Call(lib.gla_qk_norm_bwd, list(range(1, 16)), qk_shape, dict(ws=None, n=0))
    assert bwd() in (6, 8)
    for i in (0, 1, 2, 3, 4, 5, 8, 9, 11, 12):
        assert bwd(i, None) == 1
    for i in (6, 7, 10, 13, 14):
        assert bwd(i, None) in (6, 8)
    assert bwd(11, at(3)) == 5 and bwd(13, at(15) + 4) == 5 and bwd(14, at(7)) == 5 and bwd(12, at(13) + 8) == 4
    assert bwd(norm=0) == 10 and bwd(d_qo=(2560, 0, 64)) == 2


def test_workspaces_that_will_not_do(lib):
    """Where there is no device they are not reached; sizes are."""
    assert lib.gla_conv_bwd_workspace_size(ctypes.byref(conv_shape())) >= 64 * 5 * 4
    assert lib.gla_conv_bwd_workspace_size(ctypes.byref(fill(conv_shape(), W=9))) == 0
    assert lib.gla_qk_norm_bwd_workspace_size(ctypes.byref(qk_shape())) >= 2 * 64 * 4
    assert lib.gla_qk_norm_bwd_workspace_size(ctypes.byref(fill(qk_shape(), norm=0))) == 0
