"""Norm of queries and keys for each head, with the rotation by position: Python binding of
``gla_qk_norm_fwd`` and ``gla_qk_norm_bwd`` (``include/gla.h`` has the contracts).

    n = x r w,   r = (mean x^2 + eps)^-1/2  (norm="rms"),  (sum x^2 + eps)^-1/2  ("l2");  n = x  ("none")

then the first R channels of each head turn in pairs by the tables cos, sin [P, R/2] (row: the
token's position): (i, i + R/2) with layout="halves", (2 i, 2 i + 1) with "pairs". q [B, T, Hq, D]
and k [B, T, Hk, D] may be strided views; the results are what ``hda_fwd`` and ``gdn_fwd`` take. As
in ``gla.py`` nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .conv import _elem
from .gla import IO_BF16, IO_F32, _QkShape, _addr, _check, _launch, _on_stream, _workspace, load_library
from .hda import _check_rows, _fail, _tensor

NORMS = {"none": 0, "rms": 1, "l2": 2}
LAYOUTS = {"halves": 0, "pairs": 1}


# The C shape of a call depends on the tensors' types, shapes and strides alone: it is checked and
# made once for each combination.
@functools.lru_cache(maxsize=512)
def _plan(norm, layout, eps, table, tensors) -> _QkShape:
    (qs, qt, dtype), (ks, kt, kd) = tensors[:2]
    _elem(dtype)
    if norm not in NORMS:
        raise ValueError(f"norm must be one of {sorted(NORMS)}")
    if layout not in LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}")
    if len(qs) != 4 or len(ks) != 4:
        raise ValueError("q and k must be [B, T, heads, D]")
    sh = _QkShape()
    sh.B, sh.T, sh.Hq, sh.D = qs
    sh.Hk = ks[2]
    if table is not None:
        sh.P, sh.R = table[0], 2 * table[1]
    want = (qs, torch.Size((sh.B, sh.T, sh.Hk, sh.D)))
    names = ("q", "k", "dqo", "dko")
    for i, (to, (shape, strides, dt)) in enumerate(zip((sh.q, sh.k, sh.d_qo, sh.d_ko), tensors)):
        _check_rows(names[i], dt, shape, strides, dtype, want[i % 2], _elem(dtype))
        if 0 not in shape:
            to.b, to.t, to.h = strides[:3]
    sh.eps = eps
    sh.norm, sh.pairs = NORMS[norm], LAYOUTS[layout]
    sh.io = IO_BF16 if dtype == torch.bfloat16 else IO_F32
    return sh


def _shape(q, k, norm, layout, eps, cos, *grads) -> _QkShape:
    key = []
    for t, n in zip((q, k) + grads, ("q", "k", "dqo", "dko")):
        _tensor(t, n)
        key.append((t.shape, t.stride(), t.dtype))
    if cos is not None:
        _tensor(cos, "cos")
        if cos.dim() != 2:
            raise ValueError("cos must be [P, R / 2]")
    # (eps by its value: a plan is not kept for a tensor that may change)
    return _plan(norm, layout, ctypes.c_float(eps).value, None if cos is None else tuple(cos.shape), tuple(key))


def _check_inputs(sh, q, k, wq, wk, cos, sin, positions):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    if k.device != dev:
        raise ValueError(f"k: on {k.device}, expected {dev}")
    for t, n in ((wq, "wq"), (wk, "wk")):
        if t is not None:
            _check(t, n, torch.float32, (sh.D,), dev)
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        _check(cos, "cos", torch.float32, (sh.P, sh.R // 2), dev)
        _check(sin, "sin", torch.float32, (sh.P, sh.R // 2), dev)
    if positions is not None:
        _check(positions, "positions", torch.int32, (sh.B, sh.T), dev)
    return dev


def qk_norm_workspace_size(q, k, cos=None, norm: str = "rms") -> int:
    """Bytes of workspace ``qk_norm_bwd`` needs for these tensors' shapes."""
    sh = _shape(q, k, norm, "halves", 0.0, cos)
    return int(load_library().gla_qk_norm_bwd_workspace_size(ctypes.byref(sh)))


def qk_norm_fwd(q, k, wq=None, wk=None, *, cos=None, sin=None, positions=None, norm: str = "rms",
                layout: str = "halves", eps: float = 1e-6, qo=None, ko=None, stream=None):
    """wq, wk: float32 [D] or None (1); cos, sin: float32 [P, R/2] or None (no rotation); positions:
    int32 [B, T], or None: each token's index. Returns (qo, ko, rq, rk), rq [B, T, Hq] and rk
    [B, T, Hk] float32 (None with norm="none"). A token whose position is not in the tables gets zeros
    and raises the device status."""
    if stream is not None:
        return _on_stream(stream, qk_norm_fwd, q, k, wq, wk, cos=cos, sin=sin, positions=positions,
                          norm=norm, layout=layout, eps=eps, qo=qo, ko=ko)
    lib = load_library()
    sh = _shape(q, k, norm, layout, eps, cos)
    dev = _check_inputs(sh, q, k, wq, wk, cos, sin, positions)
    if qo is None:
        qo = torch.empty(q.shape, dtype=q.dtype, device=dev)
    else:
        _check(qo, "qo", q.dtype, q.shape, dev)
    if ko is None:
        ko = torch.empty(k.shape, dtype=q.dtype, device=dev)
    else:
        _check(ko, "ko", q.dtype, k.shape, dev)
    rq = rk = None
    if sh.norm:
        rq = torch.empty(q.shape[:3], dtype=torch.float32, device=dev)
        rk = torch.empty(k.shape[:3], dtype=torch.float32, device=dev)
    rc = _launch(lib.gla_qk_norm_fwd, dev, _addr(q), _addr(k), _addr(wq), _addr(wk), _addr(cos),
                 _addr(sin), _addr(positions), _addr(qo), _addr(ko), _addr(rq), _addr(rk),
                 ctypes.byref(sh))
    _fail(lib, rc, "gla_qk_norm_fwd")
    return qo, ko, rq, rk


def qk_norm_bwd(dqo, dko, q, k, rq, rk, wq=None, wk=None, *, cos=None, sin=None, positions=None,
                norm: str = "rms", layout: str = "halves", workspace=None, stream=None):
    """Gradients of ``qk_norm_fwd`` from its rq and rk (None with norm="none"). Returns (dq, dk,
    dwq | None, dwk | None): float32 [D] sums for the weights that are given."""
    if stream is not None:
        return _on_stream(stream, qk_norm_bwd, dqo, dko, q, k, rq, rk, wq, wk, cos=cos, sin=sin,
                          positions=positions, norm=norm, layout=layout, workspace=workspace)
    lib = load_library()
    sh = _shape(q, k, norm, layout, 0.0, cos, dqo, dko)
    dev = _check_inputs(sh, q, k, wq, wk, cos, sin, positions)
    for t, n in ((dqo, "dqo"), (dko, "dko")):
        if t.device != dev:
            raise ValueError(f"{n}: on {t.device}, expected {dev}")
    if sh.norm:
        _check(rq, "rq", torch.float32, q.shape[:3], dev)
        _check(rk, "rk", torch.float32, k.shape[:3], dev)
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dk = torch.empty(k.shape, dtype=q.dtype, device=dev)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    ws, nws = _workspace(workspace, dev)
    rc = _launch(lib.gla_qk_norm_bwd, dev, _addr(dqo), _addr(dko), _addr(q), _addr(k), _addr(rq),
                 _addr(rk), _addr(wq), _addr(wk), _addr(cos), _addr(sin), _addr(positions), _addr(dq),
                 _addr(dk), _addr(dwq), _addr(dwk), ctypes.byref(sh), ws, nws)
    _fail(lib, rc, "gla_qk_norm_bwd")
    return dq, dk, dwq, dwk
