"""Linear attention with one decay per head: Python binding of ``hda_fwd``, ``hda_bwd`` and
``hda_step`` (``include/gla.h`` has the contracts).

    S_t = e^decay S_{t-1} + k_t^T v_t,    o_t = scale q_t S_t

q [B,T,Hq,Dk], k [B,T,Hk,Dk] and v [B,T,Hv,Dv] may share heads (each head count divides the
number of states H = ``decay.numel()``) and may be strided views whose last dimension is
contiguous, such as slices of one projection. As in ``gla.py`` nothing is computed here.
"""
from __future__ import annotations

import ctypes

import torch

from .gla import (GLA_OK, GLAError, IO_BF16, IO_F32, _HdaShape, _check, _ptr, _stream_handle,
                  load_library, options)


def _check_rows(t, name, dtype, shape, device, align):
    """A tensor whose last dimension is contiguous and whose other strides are positive and
    multiples of ``align`` bytes (those of dimensions with more than one element)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.numel() == 0:
        return
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    for n, s in zip(t.shape[:-1], t.stride()[:-1]):
        if n > 1 and (s <= 0 or s * t.element_size() % align):
            raise ValueError(f"{name}: strides {t.stride()} must be positive multiples of "
                             f"{align} bytes")


def _strides(dst, t, dims):
    for n, s in zip(dims, t.stride()):
        setattr(dst, n, s if t.numel() else 0)


def _shape(q, k, v, H, step=False) -> _HdaShape:
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    if q.dim() != (3 if step else 4) or k.dim() != q.dim() or v.dim() != q.dim():
        raise ValueError("q, k, v must be " + ("[B, heads, D]" if step else "[B, T, heads, D]"))
    sh = _HdaShape()
    sh.B, sh.T = q.shape[0], 1 if step else q.shape[1]
    sh.H, sh.Hq, sh.Hk, sh.Hv = H, q.shape[-2], k.shape[-2], v.shape[-2]
    sh.Dk, sh.Dv = q.shape[-1], v.shape[-1]
    sh.io = IO_BF16 if q.dtype == torch.bfloat16 else IO_F32
    for n, t in (("q", q), ("k", k), ("v", v)):
        _strides(getattr(sh, n), t, "bh" if step else "bth")
    return sh


def _check_inputs(q, k, v, decay, step=False):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    align = q.element_size() if step else 16
    lead = tuple(q.shape[:-2])
    _check_rows(q, "q", q.dtype, q.shape, dev, align)
    _check_rows(k, "k", q.dtype, lead + (k.shape[-2], q.shape[-1]), dev, align)
    _check_rows(v, "v", q.dtype, lead + (v.shape[-2], v.shape[-1]), dev, align)
    _check(decay, "decay", torch.float32, (decay.numel(),), dev)
    return dev


def _state(t, name, shape, dev):
    if t is not None:
        _check(t, name, torch.float32, shape, dev)
    return t


def _fail(lib, rc, where):
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc in (6, 9) else ""
        raise GLAError(rc, where, detail)


def hda_fwd(q, k, v, decay, scale: float, h0=None, *, o=None, hT=None, return_state: bool = False,
            path: str = "auto", seq_splits: int = 0, workspace=None, stream=None):
    """Forward pass over whole sequences. decay: float32 [H] log-decays (a constant of the
    layer); h0: [B,H,Dk,Dv] float32 or None. Returns (o [B,T,H,Dv], hT | None), o in q's dtype,
    the final state hT (float32) when ``return_state`` or ``hT`` is given. Asynchronous on
    ``stream`` (default: torch's current stream)."""
    lib = load_library()
    H = decay.numel()
    sh = _shape(q, k, v, H)
    dev = _check_inputs(q, k, v, decay)
    B, T, Dk, Dv = sh.B, sh.T, sh.Dk, sh.Dv
    _state(h0, "h0", (B, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (B, T, H, Dv), dev)
    if hT is None and return_state:
        hT = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    _state(hT, "hT", (B, H, Dk, Dv), dev)
    opt = options(path, seq_splits, workspace)
    with torch.cuda.device(dev):
        rc = lib.hda_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), ctypes.c_float(scale), _ptr(h0),
                         _ptr(o), _ptr(hT), ctypes.byref(sh), ctypes.byref(opt),
                         _stream_handle(stream))
    _fail(lib, rc, "hda_fwd")
    return o, hT


def hda_bwd(do, q, k, v, decay, scale: float, h0=None, dhT=None, *, path: str = "auto",
            seq_splits: int = 0, workspace=None, stream=None):
    """Gradients of ``hda_fwd``: do is that of o, dhT that of hT (None: zero), h0 what the
    forward started from. Returns (dq, dk, dv, dh0), dh0 only when h0 is given (else None). The
    gradients of shared heads are summed in fp32."""
    lib = load_library()
    H = decay.numel()
    sh = _shape(q, k, v, H)
    dev = _check_inputs(q, k, v, decay)
    B, T, Dk, Dv = sh.B, sh.T, sh.Dk, sh.Dv
    _check_rows(do, "do", q.dtype, (B, T, H, Dv), dev, 16)
    _strides(sh.d_o, do, "bth")
    _state(h0, "h0", (B, H, Dk, Dv), dev)
    _state(dhT, "dhT", (B, H, Dk, Dv), dev)
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v))
    dh0 = None if h0 is None else torch.empty_like(h0)
    opt = options(path, seq_splits, workspace)
    with torch.cuda.device(dev):
        rc = lib.hda_bwd(_ptr(do), _ptr(q), _ptr(k), _ptr(v), _ptr(decay), ctypes.c_float(scale),
                         _ptr(h0), _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dh0),
                         ctypes.byref(sh), ctypes.byref(opt), _stream_handle(stream))
    _fail(lib, rc, "hda_bwd")
    return dq, dk, dv, dh0


def hda_workspace_size(q, k, v, decay, backward: bool = False, path: str = "auto",
                       seq_splits: int = 0) -> int:
    """Bytes of workspace ``hda_fwd`` (or ``hda_bwd``) needs for these tensors' shapes."""
    lib = load_library()
    f = lib.hda_bwd_workspace_size if backward else lib.hda_fwd_workspace_size
    return int(f(ctypes.byref(_shape(q, k, v, decay.numel())),
                 ctypes.byref(options(path, seq_splits))))


def hda_path_for(q, k, v, decay, path: str = "auto") -> str | None:
    """The path ``hda_fwd`` and ``hda_bwd`` run for these shapes ("exact" / "tc"), or None."""
    r = load_library().hda_path_for(ctypes.byref(_shape(q, k, v, decay.numel())),
                                    ctypes.byref(options(path)))
    return {1: "exact", 2: "tc"}.get(int(r))


def hda_step(q, k, v, decay, scale: float, S, slots=None, *, o=None, stream=None):
    """One token for each of R rows: q [R,Hq,Dk], k [R,Hk,Dk], v [R,Hv,Dv]. S [P,H,Dk,Dv]
    float32 is a pool of states, updated in place; row r uses page ``slots[r]`` (int32 on the
    device, each page at most once; negative: an empty row, whose output is zero), or page r
    when ``slots`` is None. Returns o [R,H,Dv] in q's dtype."""
    lib = load_library()
    H = decay.numel()
    sh = _shape(q, k, v, H, step=True)
    dev = _check_inputs(q, k, v, decay, step=True)
    R, Dk, Dv = sh.B, sh.Dk, sh.Dv
    P = S.shape[0]
    _check(S, "S", torch.float32, (P, H, Dk, Dv), dev)
    if slots is not None:
        _check(slots, "slots", torch.int32, (R,), dev)
    if o is None:
        o = torch.empty((R, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (R, H, Dv), dev)
    with torch.cuda.device(dev):
        rc = lib.hda_step(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), ctypes.c_float(scale), _ptr(S),
                          _ptr(slots), _ptr(o), P, ctypes.byref(sh), _stream_handle(stream))
    _fail(lib, rc, "hda_step")
    return o
