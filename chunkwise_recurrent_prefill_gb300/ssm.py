"""Selective state space scan: Python binding of ``ssm_fwd``, ``ssm_bwd`` and ``ssm_step``
(``include/gla.h`` has the contracts).

    d = softplus(dt + dt_bias)                       (or dt + dt_bias)
    h_t = e^(d_t A) h_{t-1} + d_t u_t B_t,    y_t = C_t . h_t + D u_t,    o_t = y_t silu(z_t)

with N states for each channel. u, dt, z [B, T, C] and Bm, Cm [B, T, G, N] (shared by the C / G
channels of a group) may be strided views, such as slices of one projection; A [C, N], D and
dt_bias [C] are float32. As in ``gla.py`` nothing is computed here.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from .conv import _elem
from .gla import (IO_BF16, IO_F32, _SsmShape, _addr, _check, _launch, _on_stream, _workspace,
                  load_library, options)
from .hda import _check_rows, _fail, _tensor

_NAMES = ("u", "dt", "z", "Bm", "Cm", "do")
_FIELDS = ("u", "dt", "z", "b", "c", "d_o")


# The C shape of a call depends on the tensors' types, shapes and strides alone: it is checked and
# made once for each combination.
@functools.lru_cache(maxsize=512)
def _plan(step, softplus, N, tensors) -> _SsmShape:
    shape, _, dtype = tensors[0]
    _elem(dtype)
    lead = 1 if step else 2
    if len(shape) != lead + 1:
        raise ValueError("u must be " + ("[R, C]" if step else "[B, T, C]"))
    C = shape[-1]
    if len(tensors[3][0]) != lead + 2:
        raise ValueError("Bm must be " + ("[R, G, N]" if step else "[B, T, G, N]"))
    G = tensors[3][0][lead]
    if N is None:
        raise ValueError("A must be [C, N]")
    sh = _SsmShape()
    sh.B, sh.T, sh.C, sh.G, sh.N = shape[0], 1 if step else shape[1], C, G, N
    for name, field, t in zip(_NAMES, _FIELDS, tensors):
        if t is None:
            continue
        tshape, strides, tdtype = t
        want = shape
        if name in ("Bm", "Cm"):
            want = torch.Size(shape[:lead] + (G, N))
            if tshape == want and G > 1 and 0 not in tshape and strides[lead] != N:
                raise ValueError(f"{name}: the groups must be contiguous")
        _check_rows(name, tdtype, tshape, strides, dtype, want, _elem(dtype))
        if 0 not in tshape:
            to = getattr(sh, field)
            to.b = strides[0]
            to.t = 0 if step else strides[1]
    sh.softplus = int(softplus)
    sh.io = IO_BF16 if dtype == torch.bfloat16 else IO_F32
    return sh


def _shape(u, dt, A, Bm, Cm, z, softplus, do=None, step=False) -> _SsmShape:
    key = []
    for n, t in zip(_NAMES, (u, dt, z, Bm, Cm, do)):
        if t is None and n in ("z", "do"):
            key.append(None)
            continue
        _tensor(t, n)
        key.append((t.shape, t.stride(), t.dtype))
    _tensor(A, "A")
    return _plan(step, bool(softplus), A.shape[1] if A.dim() == 2 else None, tuple(key))


def _check_inputs(sh, u, dt, A, Bm, Cm, D, z, dt_bias):
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t, n in ((dt, "dt"), (Bm, "Bm"), (Cm, "Cm"), (z, "z")):
        if t is not None and t.device != dev:
            raise ValueError(f"{n}: on {t.device}, expected {dev}")
    _check(A, "A", torch.float32, (sh.C, sh.N), dev)
    for t, n in ((D, "D"), (dt_bias, "dt_bias")):
        if t is not None:
            _check(t, n, torch.float32, (sh.C,), dev)
    return dev


def _state(t, name, sh, dev):
    if t is not None:
        _check(t, name, torch.float32, (sh.B, sh.C, sh.N), dev)


def ssm_workspace_size(u, dt, A, Bm, Cm, z=None, backward: bool = False, seq_splits: int = 0) -> int:
    """Bytes of workspace that are enough for ``ssm_fwd`` (or ``ssm_bwd``) with tensors of these shapes, whatever
    their alignment."""
    lib = load_library()
    f = lib.ssm_bwd_workspace_size if backward else lib.ssm_fwd_workspace_size
    return int(f(ctypes.byref(_shape(u, dt, A, Bm, Cm, z, False)),
                 ctypes.byref(options("auto", seq_splits))))


def ssm_fwd(u, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, h0=None, softplus: bool = True,
            o=None, hT=None, return_state: bool = False, seq_splits: int = 0, workspace=None,
            stream=None):
    """Whole sequences from the states h0 [B, C, N] float32 (None: zero). Returns (o [B, T, C], hT |
    None), o in u's dtype, the final states hT when ``return_state`` or ``hT`` is given."""
    if stream is not None:
        return _on_stream(stream, ssm_fwd, u, dt, A, Bm, Cm, D=D, z=z, dt_bias=dt_bias, h0=h0,
                          softplus=softplus, o=o, hT=hT, return_state=return_state,
                          seq_splits=seq_splits, workspace=workspace)
    lib = load_library()
    sh = _shape(u, dt, A, Bm, Cm, z, softplus)
    dev = _check_inputs(sh, u, dt, A, Bm, Cm, D, z, dt_bias)
    _state(h0, "h0", sh, dev)
    if o is None:
        o = torch.empty(u.shape, dtype=u.dtype, device=dev)
    else:
        _check(o, "o", u.dtype, u.shape, dev)
    if hT is None and return_state:
        hT = torch.empty((sh.B, sh.C, sh.N), dtype=torch.float32, device=dev)
    _state(hT, "hT", sh, dev)
    _workspace(workspace, dev)
    opt = options("auto", seq_splits, workspace)
    rc = _launch(lib.ssm_fwd, dev, _addr(u), _addr(dt), _addr(A), _addr(Bm), _addr(Cm), _addr(D),
                 _addr(z), _addr(dt_bias), _addr(h0), _addr(o), _addr(hT), ctypes.byref(sh),
                 ctypes.byref(opt))
    _fail(lib, rc, "ssm_fwd")
    return o, hT


def ssm_bwd(do, u, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, h0=None, dhT=None,
            softplus: bool = True, seq_splits: int = 0, workspace=None, stream=None):
    """Gradients of ``ssm_fwd``: do is that of o, dhT that of hT (None: zero). Returns (du, ddt, dA,
    dBm, dCm, dD, dz, ddt_bias, dh0), None for what was not given (dD, dz, ddt_bias, dh0). Sums over
    channels, tokens and batch entries are in fp32."""
    if stream is not None:
        return _on_stream(stream, ssm_bwd, do, u, dt, A, Bm, Cm, D=D, z=z, dt_bias=dt_bias, h0=h0,
                          dhT=dhT, softplus=softplus, seq_splits=seq_splits, workspace=workspace)
    lib = load_library()
    _tensor(do, "do")
    sh = _shape(u, dt, A, Bm, Cm, z, softplus, do)
    dev = _check_inputs(sh, u, dt, A, Bm, Cm, D, z, dt_bias)
    if do.device != dev:
        raise ValueError(f"do: on {do.device}, expected {dev}")
    _state(h0, "h0", sh, dev)
    _state(dhT, "dhT", sh, dev)
    du, ddt, dBm, dCm = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (u, dt, Bm, Cm))
    dz = None if z is None else torch.empty(z.shape, dtype=z.dtype, device=dev)
    dA = torch.empty_like(A)
    dD, dbias, dh0 = (None if t is None else torch.empty_like(t) for t in (D, dt_bias, h0))
    _workspace(workspace, dev)
    opt = options("auto", seq_splits, workspace)
    rc = _launch(lib.ssm_bwd, dev, _addr(do), _addr(u), _addr(dt), _addr(A), _addr(Bm), _addr(Cm),
                 _addr(D), _addr(z), _addr(dt_bias), _addr(h0), _addr(dhT), _addr(du), _addr(ddt),
                 _addr(dA), _addr(dBm), _addr(dCm), _addr(dD), _addr(dz), _addr(dbias), _addr(dh0),
                 ctypes.byref(sh), ctypes.byref(opt))
    _fail(lib, rc, "ssm_bwd")
    return du, ddt, dA, dBm, dCm, dD, dz, dbias, dh0


def ssm_step(u, dt, A, Bm, Cm, S, slots=None, *, D=None, z=None, dt_bias=None,
             softplus: bool = True, o=None, stream=None):
    """One token for each of R rows: u, dt, z [R, C], Bm, Cm [R, G, N]. S [P, C, N] float32 is a pool
    of states, updated in place; row r uses page ``slots[r]`` (int32 on the device, each page at
    most once; negative: an empty row, whose output is zero), or page r when ``slots`` is None.
    Returns o [R, C] in u's dtype."""
    if stream is not None:
        return _on_stream(stream, ssm_step, u, dt, A, Bm, Cm, S, slots, D=D, z=z, dt_bias=dt_bias,
                          softplus=softplus, o=o)
    lib = load_library()
    sh = _shape(u, dt, A, Bm, Cm, z, softplus, step=True)
    dev = _check_inputs(sh, u, dt, A, Bm, Cm, D, z, dt_bias)
    _tensor(S, "S")
    P = S.shape[0] if S.dim() else 0
    _check(S, "S", torch.float32, (P, sh.C, sh.N), dev)
    if slots is not None:
        _check(slots, "slots", torch.int32, (sh.B,), dev)
    if o is None:
        o = torch.empty(u.shape, dtype=u.dtype, device=dev)
    else:
        _check(o, "o", u.dtype, u.shape, dev)
    rc = _launch(lib.ssm_step, dev, _addr(u), _addr(dt), _addr(A), _addr(Bm), _addr(Cm), _addr(D),
                 _addr(z), _addr(dt_bias), _addr(S), _addr(slots), _addr(o), P, ctypes.byref(sh))
    _fail(lib, rc, "ssm_step")
    return o
