"""Short causal convolution: Python binding of ``gla_conv_fwd``, ``gla_conv_bwd`` and
``gla_conv_step`` (``include/gla.h`` has the contracts).

    y[t, c] = act(bias[c] + sum_j w[c, j] x[t - (W - 1) + j, c])

x [B, T, C] may be a strided view whose channels are contiguous, such as half of a projection. The
inputs before the first token are s0 [B, W-1, C], oldest first; a pool of such states has the
pages [P, W-1, C]. As in ``gla.py`` nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .gla import (IO_BF16, IO_F32, _ConvShape, _addr, _check, _launch, _on_stream, _workspace,
                  load_library)
from .hda import _check_rows, _fail, _tensor
from .norm import ACTS


def _elem(dtype):
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("tensors must be bfloat16 or float32")
    return 2 if dtype == torch.bfloat16 else 4


def _rows(to, name, shape, strides, dtype, want_dtype, want_shape):
    """Checks a strided [B, T, ...] (or [B, ...] of one token: ``to`` then has no t) and notes its
    strides."""
    _check_rows(name, dtype, shape, strides, want_dtype, want_shape, _elem(want_dtype))
    if 0 in shape:
        return
    to.b = strides[0]
    to.t = strides[1]


# The C shape of a call depends on the tensors' types, shapes and strides alone: it is checked and
# made once for each combination.
@functools.lru_cache(maxsize=512)
def _plan(step, act, W, x, dy) -> _ConvShape:
    shape, strides, dtype = x
    _elem(dtype)
    if len(shape) != (2 if step else 3):
        raise ValueError("x must be " + ("[R, C]" if step else "[B, T, C]"))
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    sh = _ConvShape()
    sh.B, sh.T, sh.C, sh.W = shape[0], 1 if step else shape[1], shape[-1], W
    if step:
        _check_rows("x", dtype, shape, strides, dtype, shape, _elem(dtype))
        sh.x.b = 0 if 0 in shape else strides[0]
    else:
        _rows(sh.x, "x", shape, strides, dtype, dtype, shape)
    if dy is not None:
        _rows(sh.dy, "dy", dy[0], dy[1], dy[2], dtype, shape)
    sh.act = ACTS[act]
    sh.io = IO_BF16 if dtype == torch.bfloat16 else IO_F32
    return sh


def _shape(x, w, act, dy=None, step=False) -> _ConvShape:
    _tensor(x, "x")
    _tensor(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [C, W]")
    key = None if dy is None else (dy.shape, dy.stride(), dy.dtype)
    return _plan(step, act, w.shape[1], (x.shape, x.stride(), x.dtype), key)


def _params(x, w, bias):
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    _check(w, "w", torch.float32, (x.shape[-1], w.shape[1]), x.device)
    if bias is not None:
        _check(bias, "bias", torch.float32, (x.shape[-1],), x.device)
    return x.device


def _state(t, name, x, W):
    if t is not None:
        _check(t, name, x.dtype, (x.shape[0], max(W - 1, 0), x.shape[2]), x.device)


def conv_workspace_size(x, w) -> int:
    """Bytes of workspace ``conv_bwd`` needs for x's shape."""
    return int(load_library().gla_conv_bwd_workspace_size(ctypes.byref(_shape(x, w, "none"))))


def conv_fwd(x, w, bias=None, s0=None, *, act: str = "none", y=None, sT=None,
             return_state: bool = False, stream=None):
    """Whole sequences. w: float32 [C, W], W from 1 to 8; bias: float32 [C] or None; s0 [B, W-1, C]
    in x's dtype or None (zeros). Returns (y, sT | None): sT, the last W-1 inputs, when
    ``return_state`` or ``sT`` is given."""
    if stream is not None:
        return _on_stream(stream, conv_fwd, x, w, bias, s0, act=act, y=y, sT=sT,
                          return_state=return_state)
    lib = load_library()
    sh = _shape(x, w, act)
    dev = _params(x, w, bias)
    _state(s0, "s0", x, sh.W)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check(y, "y", x.dtype, x.shape, dev)
    if sT is None and return_state:
        sT = torch.empty((sh.B, max(sh.W - 1, 0), sh.C), dtype=x.dtype, device=dev)
    _state(sT, "sT", x, sh.W)
    rc = _launch(lib.gla_conv_fwd, dev, _addr(x), _addr(w), _addr(bias), _addr(s0), _addr(y),
                 _addr(sT), ctypes.byref(sh))
    _fail(lib, rc, "gla_conv_fwd")
    return y, sT


def conv_bwd(dy, x, w, bias=None, s0=None, dsT=None, *, act: str = "none", workspace=None,
             stream=None):
    """Gradients of ``conv_fwd``: dy is that of y, dsT that of sT (None: zero). Returns (dx, dw,
    dbias | None, ds0 | None): float32 sums dw [C, W] and dbias [C] (with a bias), ds0 when s0 is
    given."""
    if stream is not None:
        return _on_stream(stream, conv_bwd, dy, x, w, bias, s0, dsT, act=act, workspace=workspace)
    lib = load_library()
    _tensor(dy, "dy")
    sh = _shape(x, w, act, dy)
    dev = _params(x, w, bias)
    if dy.device != dev:
        raise ValueError(f"dy: on {dy.device}, expected {dev}")
    _state(s0, "s0", x, sh.W)
    _state(dsT, "dsT", x, sh.W)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = torch.empty_like(w)
    db = None if bias is None else torch.empty_like(bias)
    ds0 = None if s0 is None else torch.empty_like(s0)
    ws, nws = _workspace(workspace, dev)
    rc = _launch(lib.gla_conv_bwd, dev, _addr(dy), _addr(x), _addr(w), _addr(bias), _addr(s0),
                 _addr(dsT), _addr(dx), _addr(dw), _addr(db), _addr(ds0), ctypes.byref(sh), ws, nws)
    _fail(lib, rc, "gla_conv_bwd")
    return dx, dw, db, ds0


def conv_step(x, w, S, slots=None, bias=None, *, act: str = "none", y=None, stream=None):
    """One token x [R, C] for each row. S [P, W-1, C] is a pool of the last inputs in x's dtype,
    updated in place; row r uses page ``slots[r]`` (int32 on the device, each page at most
    once; negative: an empty row, whose output is zero), or page r when ``slots`` is None. Returns
    y [R, C]."""
    if stream is not None:
        return _on_stream(stream, conv_step, x, w, S, slots, bias, act=act, y=y)
    lib = load_library()
    sh = _shape(x, w, act, step=True)
    dev = _params(x, w, bias)
    _tensor(S, "S")
    P = S.shape[0] if S.dim() else 0
    _check(S, "S", x.dtype, (P, max(sh.W - 1, 0), sh.C), dev)
    if slots is not None:
        _check(slots, "slots", torch.int32, (sh.B,), dev)
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check(y, "y", x.dtype, x.shape, dev)
    rc = _launch(lib.gla_conv_step, dev, _addr(x), _addr(w), _addr(bias), _addr(S), _addr(slots),
                 _addr(y), P, ctypes.byref(sh))
    _fail(lib, rc, "gla_conv_step")
    return y
