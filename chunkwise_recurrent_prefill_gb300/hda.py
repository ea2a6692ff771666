"""Linear attention with one decay per head: Python binding of ``hda_fwd``, ``hda_bwd`` and
``hda_step`` (``include/gla.h`` has the contracts).

    S_t = e^decay S_{t-1} + k_t^T v_t,    o_t = scale q_t S_t

q [B,T,Hq,Dk], k [B,T,Hk,Dk] and v [B,T,Hv,Dv] may share heads (each head count divides the
number of states H = ``decay.numel()``) and may be strided views whose last dimension is
contiguous, such as slices of one projection. As in ``gla.py`` nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .gla import (GLA_OK, GLAError, IO_BF16, IO_F32, _HdaShape, _check, _addr, _launch,
                  _on_stream, _workspace, load_library, options)


def _check_rows(name, dtype, shape, strides, want_dtype, want_shape, align):
    """The last dimension is contiguous and the strides of the others (those with more than one
    element) are positive multiples of ``align`` bytes."""
    if dtype != want_dtype:
        raise TypeError(f"{name}: dtype {dtype}, expected {want_dtype}")
    if shape != want_shape:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {tuple(want_shape)}")
    if 0 in shape:
        return
    if shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    es = 2 if dtype == torch.bfloat16 else 4
    for n, s in zip(shape[:-1], strides[:-1]):
        if n > 1 and (s <= 0 or s * es % align):
            raise ValueError(f"{name}: strides {tuple(strides)} must be positive multiples of "
                             f"{align} bytes")


# The C shape of a call depends on the tensors' types, shapes and strides alone: it is checked and
# made once for each combination.
@functools.lru_cache(maxsize=512)
def _plan(step, H, dtype, tensors) -> _HdaShape:
    (qs, qt, _), (ks, kt, kd), (vs, vt, vd) = tensors[:3]
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    dims = 3 if step else 4
    if len(qs) != dims or len(ks) != dims or len(vs) != dims:
        raise ValueError("q, k, v must be " + ("[B, heads, D]" if step else "[B, T, heads, D]"))
    align = (2 if dtype == torch.bfloat16 else 4) if step else 16
    lead = qs[:-2]
    _check_rows("q", dtype, qs, qt, dtype, qs, align)
    _check_rows("k", kd, ks, kt, dtype, torch.Size(lead + (ks[-2], qs[-1])), align)
    _check_rows("v", vd, vs, vt, dtype, torch.Size(lead + (vs[-2], vs[-1])), align)
    sh = _HdaShape()
    sh.B, sh.T = qs[0], 1 if step else qs[1]
    sh.H, sh.Hq, sh.Hk, sh.Hv = H, qs[-2], ks[-2], vs[-2]
    sh.Dk, sh.Dv = qs[-1], vs[-1]
    sh.io = IO_BF16 if dtype == torch.bfloat16 else IO_F32
    rows = [("q", qs, qt), ("k", ks, kt), ("v", vs, vt)]
    if len(tensors) > 3:
        os, ot, od = tensors[3]
        _check_rows("do", od, os, ot, dtype, torch.Size((sh.B, sh.T, H, sh.Dv)), align)
        rows.append(("d_o", os, ot))
    for n, shape, strides in rows:
        for d, s in zip("bh" if step else "bth", strides):
            setattr(getattr(sh, n), d, 0 if 0 in shape else s)
    return sh


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")


def _shape(q, k, v, decay, do=None, step=False):
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (decay, "decay")):
        _tensor(t, n)
    ts = ((q.shape, q.stride(), q.dtype), (k.shape, k.stride(), k.dtype), (v.shape, v.stride(), v.dtype))
    if do is not None:
        ts += ((do.shape, do.stride(), do.dtype),)
    return _plan(step, decay.numel(), q.dtype, ts)


def _check_inputs(q, k, v, decay):
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t, n in ((k, "k"), (v, "v")):
        if t.device != dev:
            raise ValueError(f"{n}: on {t.device}, expected {dev}")
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
    ``stream`` (default: torch's current stream), which the new outputs belong to."""
    if stream is not None:
        return _on_stream(stream, hda_fwd, q, k, v, decay, scale, h0, o=o, hT=hT,
                          return_state=return_state, path=path, seq_splits=seq_splits,
                          workspace=workspace)
    lib = load_library()
    sh = _shape(q, k, v, decay)
    dev = _check_inputs(q, k, v, decay)
    B, T, H, Dk, Dv = sh.B, sh.T, sh.H, sh.Dk, sh.Dv
    _state(h0, "h0", (B, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (B, T, H, Dv), dev)
    if hT is None and return_state:
        hT = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    _state(hT, "hT", (B, H, Dk, Dv), dev)
    _workspace(workspace, dev)
    opt = options(path, seq_splits, workspace)
    rc = _launch(lib.hda_fwd, dev, _addr(q), _addr(k), _addr(v), _addr(decay), scale, _addr(h0),
                 _addr(o), _addr(hT), ctypes.byref(sh), ctypes.byref(opt))
    _fail(lib, rc, "hda_fwd")
    return o, hT


def hda_bwd(do, q, k, v, decay, scale: float, h0=None, dhT=None, *, path: str = "auto",
            seq_splits: int = 0, workspace=None, stream=None):
    """Gradients of ``hda_fwd``: do is that of o, dhT that of hT (None: zero), h0 what the
    forward started from. Returns (dq, dk, dv, dh0), dh0 only when h0 is given (else None). The
    gradients of shared heads are summed in fp32."""
    if stream is not None:
        return _on_stream(stream, hda_bwd, do, q, k, v, decay, scale, h0, dhT, path=path,
                          seq_splits=seq_splits, workspace=workspace)
    lib = load_library()
    _tensor(do, "do")
    sh = _shape(q, k, v, decay, do)
    dev = _check_inputs(q, k, v, decay)
    if do.device != dev:
        raise ValueError(f"do: on {do.device}, expected {dev}")
    B, H, Dk, Dv = sh.B, sh.H, sh.Dk, sh.Dv
    _state(h0, "h0", (B, H, Dk, Dv), dev)
    _state(dhT, "dhT", (B, H, Dk, Dv), dev)
    dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k, v))
    dh0 = None if h0 is None else torch.empty_like(h0)
    _workspace(workspace, dev)
    opt = options(path, seq_splits, workspace)
    rc = _launch(lib.hda_bwd, dev, _addr(do), _addr(q), _addr(k), _addr(v), _addr(decay), scale,
                 _addr(h0), _addr(dhT), _addr(dq), _addr(dk), _addr(dv), _addr(dh0), ctypes.byref(sh),
                 ctypes.byref(opt))
    _fail(lib, rc, "hda_bwd")
    return dq, dk, dv, dh0


def hda_workspace_size(q, k, v, decay, backward: bool = False, path: str = "auto",
                       seq_splits: int = 0) -> int:
    """Bytes of workspace ``hda_fwd`` (or ``hda_bwd``) needs for these tensors' shapes."""
    lib = load_library()
    f = lib.hda_bwd_workspace_size if backward else lib.hda_fwd_workspace_size
    return int(f(ctypes.byref(_shape(q, k, v, decay)),
                 ctypes.byref(options(path, seq_splits))))


def hda_path_for(q, k, v, decay, path: str = "auto") -> str | None:
    """The path ``hda_fwd`` and ``hda_bwd`` run for these shapes ("exact" / "tc"), or None."""
    r = load_library().hda_path_for(ctypes.byref(_shape(q, k, v, decay)),
                                    ctypes.byref(options(path)))
    return {1: "exact", 2: "tc"}.get(int(r))


def hda_step(q, k, v, decay, scale: float, S, slots=None, *, o=None, stream=None):
    """One token for each of R rows: q [R,Hq,Dk], k [R,Hk,Dk], v [R,Hv,Dv]. S [P,H,Dk,Dv]
    float32 is a pool of states, updated in place; row r uses page ``slots[r]`` (int32 on the
    device, each page at most once; negative: an empty row, whose output is zero), or page r
    when ``slots`` is None. Returns o [R,H,Dv] in q's dtype."""
    if stream is not None:
        return _on_stream(stream, hda_step, q, k, v, decay, scale, S, slots, o=o)
    lib = load_library()
    sh = _shape(q, k, v, decay, step=True)
    dev = _check_inputs(q, k, v, decay)
    R, H, Dk, Dv = sh.B, sh.H, sh.Dk, sh.Dv
    _tensor(S, "S")
    P = S.shape[0] if S.dim() else 0
    _check(S, "S", torch.float32, (P, H, Dk, Dv), dev)
    if slots is not None:
        _check(slots, "slots", torch.int32, (R,), dev)
    if o is None:
        o = torch.empty((R, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (R, H, Dv), dev)
    rc = _launch(lib.hda_step, dev, _addr(q), _addr(k), _addr(v), _addr(decay), scale, _addr(S),
                 _addr(slots), _addr(o), P, ctypes.byref(sh))
    _fail(lib, rc, "hda_step")
    return o
