"""Group norm with an activation, channels last: Python binding of ``gla_group_norm_fwd`` and
``gla_group_norm_bwd`` (``include/gla.h`` has the contracts).

x is [N, ..., C]: the statistics are taken over the middle dimensions and the C / groups channels
of each group. The norm over each head of a token is x [B T, C] with one group per head.
"""
from __future__ import annotations

import ctypes

import torch

from .gla import IO_BF16, IO_F32, _NormShape, _check, _ptr, _stream_handle, load_library
from .hda import _fail

ACTS = {"none": 0, "silu": 1, "gelu": 2}


def _rows(t, name, dtype, shape, dev):
    """(stride of N, stride of a position) of [N, ..., C]; the positions must be evenly spaced."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    if t.numel() == 0:
        return 0, 0
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the channels must be contiguous")
    step, run = 0, 1      # stride of one position, positions covered so far
    for n, s in zip(reversed(t.shape[1:-1]), reversed(t.stride()[1:-1])):
        if n == 1:
            continue
        if step and s != step * run:
            raise ValueError(f"{name}: the positions must be evenly spaced in memory")
        step = step or s
        run *= n
    sn = t.stride(0) if t.shape[0] > 1 else max(step, t.shape[-1]) * run
    sl = step or t.shape[-1]
    if sn <= 0 or sl <= 0:
        raise ValueError(f"{name}: strides {t.stride()} must be positive")
    return sn, sl


def _shape(x, groups, eps, act, gate, dy=None) -> _NormShape:
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be bfloat16 or float32")
    if x.dim() < 2:
        raise ValueError("x must be [N, ..., C]")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    sh = _NormShape()
    sh.N, sh.C, sh.G = x.shape[0], x.shape[-1], int(groups)
    sh.L = 1
    for n in x.shape[1:-1]:
        sh.L *= n
    sh.x_n, sh.x_l = _rows(x, "x", x.dtype, x.shape, x.device)
    if gate is not None:
        sh.gate_n, sh.gate_l = _rows(gate, "gate", x.dtype, x.shape, x.device)
    if dy is not None:
        sh.dy_n, sh.dy_l = _rows(dy, "dy", x.dtype, x.shape, x.device)
    sh.eps, sh.act = eps, ACTS[act]
    sh.io = IO_BF16 if x.dtype == torch.bfloat16 else IO_F32
    return sh


def _affine(x, weight, bias):
    if x.device.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _check(t, n, torch.float32, (x.shape[-1],), x.device)


def _workspace(workspace, dev):
    if workspace is None:
        return None, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def group_norm_workspace_size(x, groups: int, backward: bool = False, gate=None) -> int:
    """Bytes of workspace the two calls need for x's shape."""
    sh = _shape(x, groups, 0.0, "none", gate)
    return int(load_library().gla_group_norm_workspace_size(ctypes.byref(sh), int(backward)))


def group_norm_fwd(x, groups: int, weight=None, bias=None, *, eps: float = 1e-5, act: str = "none",
                   gate=None, y=None, workspace=None, stream=None):
    """y = act(u), or u act(gate) with a gate, of u = (x - mean) rstd weight + bias. weight, bias:
    float32 [C] or None. Returns (y, mean [N, groups], rstd [N, groups])."""
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
    with torch.cuda.device(dev):
        rc = lib.gla_group_norm_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(gate), _ptr(y),
                                    _ptr(mean), _ptr(rstd), ctypes.byref(sh), ws, nws,
                                    _stream_handle(stream))
    _fail(lib, rc, "gla_group_norm_fwd")
    return y, mean, rstd


def group_norm_bwd(dy, x, mean, rstd, groups: int, weight=None, bias=None, *, act: str = "none",
                   gate=None, workspace=None, stream=None):
    """Gradients of ``group_norm_fwd`` from its mean and rstd. Returns (dx, dweight | None,
    dbias | None, dgate | None): float32 [C] sums for the parameters that are given."""
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
    with torch.cuda.device(dev):
        rc = lib.gla_group_norm_bwd(_ptr(dy), _ptr(x), _ptr(mean), _ptr(rstd), _ptr(weight),
                                    _ptr(bias), _ptr(gate), _ptr(dx), _ptr(dw), _ptr(db), _ptr(dz),
                                    ctypes.byref(sh), ws, nws, _stream_handle(stream))
    _fail(lib, rc, "gla_group_norm_bwd")
    return dx, dw, db, dz
