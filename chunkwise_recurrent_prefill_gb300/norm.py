"""Group norm with an activation, channels last: Python binding of ``gla_group_norm_fwd`` and
``gla_group_norm_bwd`` (``include/gla.h`` has the contracts).

x is [N, ..., C]: the statistics are taken over the middle dimensions and the C / groups channels
of each group. The norm over each head of a token is x [B T, C] with one group per head.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from .gla import IO_BF16, IO_F32, _NormShape, _check, _addr, _launch, _on_stream, _workspace, load_library
from .hda import _fail

ACTS = {"none": 0, "silu": 1, "gelu": 2}


def _rows(name, dtype, shape, strides, want_dtype, want_shape):
    """(stride of N, stride of a position) of [N, ..., C]; the positions must be evenly spaced."""
    if dtype != want_dtype:
        raise TypeError(f"{name}: dtype {dtype}, expected {want_dtype}")
    if shape != want_shape:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {tuple(want_shape)}")
    if 0 in shape:
        return 0, 0
    if shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    step, run = 0, 1      # stride of one position, positions covered so far
    for n, s in zip(reversed(shape[1:-1]), reversed(strides[1:-1])):
        if n == 1:
            continue
        if s <= 0:
            raise ValueError(f"{name}: strides {tuple(strides)} must be positive")
        if step and s != step * run:
            raise ValueError(f"{name}: the positions must be evenly spaced in memory")
        step = step or s
        run *= n
    sn = strides[0] if shape[0] > 1 else max(step, shape[-1]) * run
    sl = step or shape[-1]
    if sn <= 0:
        raise ValueError(f"{name}: strides {tuple(strides)} must be positive")
    return sn, sl


# The C shape of a call depends on the tensors' types, shapes and strides alone: it is checked and
# made once for each combination.
@functools.lru_cache(maxsize=512)
def _plan(groups, eps, act, x, gate, dy) -> _NormShape:
    shape, strides, dtype = x
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be bfloat16 or float32")
    if len(shape) < 2:
        raise ValueError("x must be [N, ..., C]")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    sh = _NormShape()
    sh.N, sh.C, sh.G = shape[0], shape[-1], groups
    sh.L = 1
    for n in shape[1:-1]:
        sh.L *= n
    sh.x_n, sh.x_l = _rows("x", dtype, shape, strides, dtype, shape)
    if gate is not None:
        sh.gate_n, sh.gate_l = _rows("gate", gate[2], gate[0], gate[1], dtype, shape)
    if dy is not None:
        sh.dy_n, sh.dy_l = _rows("dy", dy[2], dy[0], dy[1], dtype, shape)
    sh.eps, sh.act = eps, ACTS[act]
    sh.io = IO_BF16 if dtype == torch.bfloat16 else IO_F32
    return sh


def _shape(x, groups, eps, act, gate, dy=None) -> _NormShape:
    key = []
    for t, n in ((x, "x"), (gate, "gate"), (dy, "dy")):
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
        if t is not None and t.device != x.device:
            raise ValueError(f"{n}: on {t.device}, expected {x.device}")
        key.append(None if t is None else (t.shape, t.stride(), t.dtype))
    # (eps by its value: a plan is not kept for a tensor that may change)
    return _plan(operator.index(groups), ctypes.c_float(eps).value, act, *key)


def _affine(x, weight, bias):
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check(t, n, torch.float32, (x.shape[-1],), x.device)


def group_norm_workspace_size(x, groups: int, backward: bool = False, gate=None) -> int:
    """Bytes of workspace the two calls need for x's shape."""
    sh = _shape(x, groups, 0.0, "none", gate)
    return int(load_library().gla_group_norm_workspace_size(ctypes.byref(sh), int(backward)))


def group_norm_fwd(x, groups: int, weight=None, bias=None, *, eps: float = 1e-5, act: str = "none",
                   gate=None, y=None, workspace=None, stream=None):
    """y = act(u), or u act(gate) with a gate, of u = (x - mean) rstd weight + bias. weight, bias:
    float32 [C] or None. Returns (y, mean [N, groups], rstd [N, groups])."""
    if stream is not None:
        return _on_stream(stream, group_norm_fwd, x, groups, weight, bias, eps=eps, act=act,
                          gate=gate, y=y, workspace=workspace)
    lib = load_library()
    sh = _shape(x, groups, eps, act, gate)
    _affine(x, weight, bias)
    dev = x.device
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _check(y, "y", x.dtype, x.shape, dev)
    mean = torch.empty((sh.N, max(sh.G, 0)), dtype=torch.float32, device=dev)
    rstd = torch.empty_like(mean)
    ws, nws = _workspace(workspace, dev)
    rc = _launch(lib.gla_group_norm_fwd, dev, _addr(x), _addr(weight), _addr(bias), _addr(gate),
                 _addr(y), _addr(mean), _addr(rstd), ctypes.byref(sh), ws, nws)
    _fail(lib, rc, "gla_group_norm_fwd")
    return y, mean, rstd


def group_norm_bwd(dy, x, mean, rstd, groups: int, weight=None, bias=None, *, act: str = "none",
                   gate=None, workspace=None, stream=None):
    """Gradients of ``group_norm_fwd`` from its mean and rstd. Returns (dx, dweight | None,
    dbias | None, dgate | None): float32 [C] sums for the parameters that are given."""
    if stream is not None:
        return _on_stream(stream, group_norm_bwd, dy, x, mean, rstd, groups, weight, bias, act=act,
                          gate=gate, workspace=workspace)
    lib = load_library()
    sh = _shape(x, groups, 0.0, act, gate, dy)
    _affine(x, weight, bias)
    dev = x.device
    for t, n in ((mean, "mean"), (rstd, "rstd")):
        _check(t, n, torch.float32, (sh.N, sh.G), dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dz = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = None if weight is None else torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    ws, nws = _workspace(workspace, dev)
    rc = _launch(lib.gla_group_norm_bwd, dev, _addr(dy), _addr(x), _addr(mean), _addr(rstd),
                 _addr(weight), _addr(bias), _addr(gate), _addr(dx), _addr(dw), _addr(db), _addr(dz),
                 ctypes.byref(sh), ws, nws)
    _fail(lib, rc, "gla_group_norm_bwd")
    return dx, dw, db, dz
