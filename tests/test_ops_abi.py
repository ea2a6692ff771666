"""Argument checks of the decay attention, group norm and page calls on fake device addresses:
every call here is refused on the host (or has nothing to launch). Run where no GPU is visible."""
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


def test_exports(lib):
    src = open(os.path.join(ROOT, "include", "gla.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"\b(hda_[a-z0-9_]+)\s*\(", src))
    assert {"hda_fwd", "hda_bwd", "hda_step", "hda_path_for"} <= names
    assert all(hasattr(lib, n) for n in names)
    assert lib.gla_status_string(12) == b"GLA_ERR_BAD_PAGES"


def shape(**kw):
    from chunkwise_recurrent_prefill_gb300.gla import _HdaShape
    sh = _HdaShape(B=1, T=128, H=4, Hq=4, Hk=2, Hv=4, Dk=128, Dv=128, io=0)
    for n, v in kw.items():
        if isinstance(v, tuple):
            s = getattr(sh, n)
            s.b, s.t, s.h = v
        else:
            setattr(sh, n, v)
    return sh


def fwd(lib, q=1 << 36, k=2 << 36, v=3 << 36, d=4 << 36, h0=None, o=5 << 36, hT=None, opt=None, **kw):
    from chunkwise_recurrent_prefill_gb300.gla import _Options
    o_ = ctypes.byref(opt) if opt is not None else ctypes.POINTER(_Options)()
    return lib.hda_fwd(vp(q), vp(k), vp(v), vp(d), 1.0, vp(h0), vp(o), vp(hT),
                       ctypes.byref(shape(**kw)), o_, None)


def test_forward_checks(lib):
    from chunkwise_recurrent_prefill_gb300.gla import _HdaShape, options
    assert fwd(lib, q=None) == 1 and fwd(lib, d=None) == 1 and fwd(lib, o=None) == 1
    assert lib.hda_fwd(None, None, None, None, 1.0, None, None, None,
                       ctypes.POINTER(_HdaShape)(), None, None) == 1
    assert fwd(lib, B=-1) == 2 and fwd(lib, T=-1) == 2 and fwd(lib, Hk=3) == 2 and fwd(lib, Hq=0) == 2
    assert fwd(lib, B=1 << 40, T=1 << 30) == 2
    assert fwd(lib, Dk=12) == 3 and fwd(lib, Dv=264) == 3 and fwd(lib, Dk=0) == 3
    assert fwd(lib, k=(2 << 36) + 8) == 4 and fwd(lib, d=(4 << 36) + 2) == 4
    assert fwd(lib) in (6, 8)                               # all in order: no device to run on
    assert fwd(lib, o=(1 << 36) + 1024) == 5                # inside q
    assert fwd(lib, h0=6 << 36, hT=6 << 36) == 5 and fwd(lib, hT=5 << 36) == 5
    assert fwd(lib, io=7) == 10 and fwd(lib, opt=options("auto", -1)) == 10
    assert fwd(lib, opt=options("auto", 0, None, "scalar")) == 10
    assert fwd(lib, io=1, opt=options("tc")) == 3 and fwd(lib, Dk=96, opt=options("tc")) == 3


def test_strides(lib):
    def call(**kw):
        sh = shape(B=2, **kw)
        return lib.hda_fwd(vp(1 << 36), vp(2 << 36), vp(3 << 36), vp(4 << 36), 1.0, None, vp(5 << 36),
                           None, ctypes.byref(sh), None, None)
    good = (128 * 2048, 2048, 128)
    assert call(q=good) in (6, 8)
    assert call(q=(128 * 2048, 2048, 124)) == 4             # heads 248 bytes apart
    assert call(q=(128 * 2048, -2048, 128)) == 4
    assert call(v=(0, 2048, 128)) == 4
    assert call(q=(128 * 2048, 1 << 60, 128)) == 2          # past what an address can be
    # a dimension of one element may say anything
    sh = shape(B=1, q=(-5, 2048, 128))
    assert lib.hda_fwd(vp(1 << 36), vp(2 << 36), vp(3 << 36), vp(4 << 36), 1.0, None, vp(5 << 36), None,
                       ctypes.byref(sh), None, None) in (6, 8)
    # o laid inside the gaps of a strided q is still an overlap
    sh = shape(B=1, q=(0, 1 << 20, 128))
    assert lib.hda_fwd(vp(1 << 36), vp(2 << 36), vp(3 << 36), vp(4 << 36), 1.0, None,
                       vp((1 << 36) + 4096), None, ctypes.byref(sh), None, None) == 5


def test_backward_checks(lib):
    base = [1, 2, 3, 4, 5, None, None, 8, 9, 10, None]      # do q k v decay h0 dhT dq dk dv dh0

    def call(i=None, value=None, **kw):
        a = [None if x is None else x << 36 for x in base]
        if i is not None:
            a[i] = value
        p = [vp(x) for x in a]
        return lib.hda_bwd(p[0], p[1], p[2], p[3], p[4], 1.0, *p[5:], ctypes.byref(shape(**kw)), None, None)

    assert call() in (6, 8)
    for i in (0, 1, 4, 7, 8, 9):
        assert call(i, None) == 1
    assert call(7, (8 << 36) + 4) == 4 and call(6, (7 << 36) + 8) == 4
    assert call(9, 8 << 36) == 5 and call(10, 4 << 36) == 5 and call(8, 2 << 36) == 5
    assert call(d_o=(0, 500, 128)) == 4
    assert call(Hv=3) == 2 and call(Dv=20) == 3


def test_step_checks(lib):
    def call(q=1 << 36, S=2 << 36, slots=3 << 36, o=4 << 36, P=4, **kw):
        sh = shape(**{"B": 2, **kw})
        return lib.hda_step(vp(q), vp(5 << 36), vp(6 << 36), vp(7 << 36), 1.0, vp(S), vp(slots), vp(o), P,
                            ctypes.byref(sh), None)
    assert call() in (6, 8)
    assert call(q=None) == 1 and call(S=None) == 1 and call(o=None) == 1
    assert call(P=-1) == 2 and call(slots=None, P=1) == 2 and call(Hq=3) == 2
    assert call(Dk=0) == 3 and call(Dv=6) == 3 and call(Dk=2000) == 3
    assert call(q=(1 << 36) + 1) == 4 and call(S=(2 << 36) + 4) == 4 and call(slots=(3 << 36) + 2) == 4
    assert call(o=2 << 36) == 5 and call(S=5 << 36) == 5
    assert call(io=2) == 10


def test_norm_checks(lib):
    from chunkwise_recurrent_prefill_gb300.gla import _NormShape

    def call(x=1 << 36, y=2 << 36, ws=None, nws=0, gate=None, **kw):
        sh = _NormShape(N=2, L=10, C=64, G=4, eps=1e-5, act=1, io=0)
        for n, v in kw.items():
            setattr(sh, n, v)
        return lib.gla_group_norm_fwd(vp(x), None, None, vp(gate), vp(y), vp(3 << 36), vp(4 << 36),
                                      ctypes.byref(sh), vp(ws), nws, None)
    assert call() in (6, 8)
    assert call(x=None) == 1 and call(y=None) == 1
    assert call(G=0) == 2 and call(G=5) == 2 and call(N=-1) == 2 and call(L=1 << 40) == 2
    assert call(x_n=640, x_l=-64) == 2
    assert call(y=(2 << 36) + 8) == 4 and call(x=(1 << 36) + 1) == 4
    assert call(y=1 << 36) == 5 and call(gate=2 << 36) == 5
    assert call(io=4) == 10 and call(act=3) == 10 and call(eps=-1.0) == 10 and call(eps=float("nan")) == 10


def test_page_checks(lib):
    pool, tab, st, cnt, a, c = (i << 36 for i in range(1, 7))

    def fork(P=8, nb=64, R=4, M=2, n=2, pool=pool, tab=tab, st=st, cnt=cnt, a=a, c=c):
        return lib.gla_pages_fork(vp(pool), P, nb, vp(tab), R, M, vp(st), vp(cnt), vp(a), vp(c), n, None)
    assert fork() in (6, 8)
    assert fork(pool=None) == 1 and fork(tab=None) == 1 and fork(cnt=None) == 1 and fork(a=None) == 1
    assert fork(P=-1) == 2 and fork(M=1 << 40) == 2 and fork(n=-2) == 2 and fork(R=1 << 20, M=1 << 20) == 2
    assert fork(nb=24) == 4 and fork(pool=pool + 8) == 4 and fork(tab=tab + 2) == 4
    assert fork(a=tab) == 5 and fork(st=tab) == 5 and fork(tab=pool + 64) == 5
    assert lib.gla_pages_copy(vp(pool), 4, 60, vp(a), vp(c), 1, None) == 4
    assert lib.gla_pages_copy(vp(pool), 4, 64, vp(pool), vp(c), 1, None) == 5
    assert lib.gla_pages_free(8, vp(tab), 4, 2, vp(st), vp(cnt), None, 1, None) == 1
    assert lib.gla_pages_free(8, vp(tab), 4, 2, vp(st), vp(cnt), vp(cnt), 1, None) == 5
    assert lib.gla_pages_compact(vp(pool), 8, 64, vp(tab), 4, 2, vp(tab), vp(cnt), None) == 5
