"""Python binding of libgla.so (argument marshalling only).

Every step of the forward pass runs inside the library's CUDA kernels; this module
checks tensor dtypes/shapes/devices, allocates outputs with torch (device memory is
plumbing here) and passes raw pointers and the current CUDA stream to the C ABI
declared in ``include/gla.h``. There is no CPU or PyTorch fallback: if the library is
missing or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libgla.so")

GLA_OK = 0
STATUS = {
    0: "GLA_OK", 1: "GLA_ERR_NULL_ARG", 2: "GLA_ERR_BAD_SHAPE", 3: "GLA_ERR_UNSUPPORTED_DIM",
    4: "GLA_ERR_MISALIGNED", 5: "GLA_ERR_ALIAS", 6: "GLA_ERR_LAUNCH",
    7: "GLA_ERR_DEVICE_TIMEOUT", 8: "GLA_ERR_UNSUPPORTED_DEVICE", 9: "GLA_ERR_WORKSPACE",
    10: "GLA_ERR_BAD_OPTION", 11: "GLA_ERR_BAD_SEQLENS", 12: "GLA_ERR_BAD_PAGES",
}
PATHS = {"auto": 0, "exact": 1, "tc": 2}
GATES = {"key": 0, "scalar": 1}
IO_BF16, IO_F32 = 0, 1


class GLAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = f"{where}: {STATUS.get(status, status)}"
        super().__init__(msg + (f" ({detail})" if detail else ""))


class _Options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("seq_splits", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("gate", ctypes.c_int)]


class _Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64), ("h", ctypes.c_int64)]


class _HdaShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "H", "Hq", "Hk", "Hv", "Dk", "Dv")] + \
        [(n, _Strides) for n in ("q", "k", "v", "d_o")] + [("io", ctypes.c_int)]


class _NormShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("N", "L", "C", "G", "x_n", "x_l", "gate_n", "gate_l",
                                              "dy_n", "dy_l")] + \
        [("eps", ctypes.c_float), ("act", ctypes.c_int), ("io", ctypes.c_int)]


class _Rows(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("t", ctypes.c_int64)]


class _ConvShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "C", "W")] + \
        [(n, _Rows) for n in ("x", "dy")] + [("act", ctypes.c_int), ("io", ctypes.c_int)]


class _SsmShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "C", "G", "N")] + \
        [(n, _Rows) for n in ("u", "dt", "z", "b", "c", "d_o")] + \
        [("softplus", ctypes.c_int), ("io", ctypes.c_int)]


class _QkShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "T", "Hq", "Hk", "D", "R", "P")] + \
        [(n, _Strides) for n in ("q", "k", "d_qo", "d_ko")] + \
        [("eps", ctypes.c_float), ("norm", ctypes.c_int), ("pairs", ctypes.c_int), ("io", ctypes.c_int)]


_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgla.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libgla.so is not built ({path}); run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            vp, i64, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float
            sig = [vp, vp, vp, vp, f32, vp, vp, vp, i64, i64, i64, i64, i64]
            lib.gla_fwd.argtypes = sig + [vp]
            lib.gla_fwd_f32.argtypes = sig + [vp]
            lib.gla_fwd_ex.argtypes = sig + [ctypes.c_int, ctypes.POINTER(_Options), vp]
            for f in (lib.gla_fwd, lib.gla_fwd_f32, lib.gla_fwd_ex):
                f.restype = ctypes.c_int
            lib.gla_step.argtypes = [vp, vp, vp, vp, f32, vp, vp, i64, i64, i64, i64,
                                     ctypes.c_int, vp]
            lib.gla_fwd_varlen.argtypes = [vp, vp, vp, vp, f32, vp, vp, vp, vp, i64, i64, i64,
                                           i64, i64, ctypes.c_int, ctypes.POINTER(_Options), vp]
            lib.gla_fwd_varlen.restype = ctypes.c_int
            lib.gla_step.restype = ctypes.c_int
            lib.gla_fwd_noalloc.argtypes = sig + [ctypes.c_int, vp]
            lib.gla_fwd_noalloc.restype = ctypes.c_int
            lib.gla_fwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, ctypes.c_int,
                                                   ctypes.POINTER(_Options)]
            lib.gla_fwd_workspace_size.restype = ctypes.c_size_t
            lib.gla_last_device_status.argtypes = [vp]
            lib.gla_last_device_status.restype = ctypes.c_int
            lib.gla_status_string.argtypes = [ctypes.c_int]
            lib.gla_status_string.restype = ctypes.c_char_p
            lib.gla_path_for.argtypes = [i64, i64, i64, i64, i64, ctypes.c_int,
                                         ctypes.POINTER(_Options)]
            lib.gla_path_for.restype = ctypes.c_int
            lib.gla_last_error_detail.argtypes = []
            lib.gla_last_error_detail.restype = ctypes.c_char_p
            lib.gla_launch_counter.argtypes = []
            lib.gla_launch_counter.restype = ctypes.c_uint64
            lib.gla_workspace_allocations.argtypes = []
            lib.gla_workspace_allocations.restype = ctypes.c_uint64
            lib.gla_version.argtypes = []
            lib.gla_version.restype = ctypes.c_int
            lib.gdn_fwd.argtypes = [vp, vp, vp, vp, vp, f32, vp, vp, vp, i64, i64, i64, i64, i64,
                                    ctypes.c_int, vp, ctypes.c_size_t, vp]
            lib.gdn_fwd.restype = ctypes.c_int
            lib.gdn_fwd_workspace_size.argtypes = [i64, i64, i64, i64, i64]
            lib.gdn_fwd_workspace_size.restype = ctypes.c_size_t
            hs, ns = ctypes.POINTER(_HdaShape), ctypes.POINTER(_NormShape)
            opt = ctypes.POINTER(_Options)
            lib.hda_fwd.argtypes = [vp, vp, vp, vp, f32, vp, vp, vp, hs, opt, vp]
            lib.hda_bwd.argtypes = [vp, vp, vp, vp, vp, f32] + [vp] * 6 + [hs, opt, vp]
            lib.hda_step.argtypes = [vp, vp, vp, vp, f32, vp, vp, vp, i64, hs, vp]
            lib.hda_path_for.argtypes = [hs, opt]
            lib.gla_group_norm_fwd.argtypes = [vp] * 7 + [ns, vp, ctypes.c_size_t, vp]
            lib.gla_group_norm_bwd.argtypes = [vp] * 11 + [ns, vp, ctypes.c_size_t, vp]
            lib.gla_pages_copy.argtypes = [vp, i64, i64, vp, vp, i64, vp]
            fork = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64]
            free = [i64, vp, i64, i64, vp, vp, vp, i64]
            compact = [vp, i64, i64, vp, i64, i64, vp, vp]
            ws = [vp, ctypes.c_size_t]
            lib.gla_pages_fork.argtypes, lib.gla_pages_fork_ex.argtypes = fork + [vp], fork + ws + [vp]
            lib.gla_pages_free.argtypes, lib.gla_pages_free_ex.argtypes = free + [vp], free + ws + [vp]
            lib.gla_pages_compact.argtypes = compact + [vp]
            lib.gla_pages_compact_ex.argtypes = compact + ws + [vp]
            for f in (lib.hda_fwd, lib.hda_bwd, lib.hda_step, lib.hda_path_for,
                      lib.gla_group_norm_fwd, lib.gla_group_norm_bwd, lib.gla_pages_copy,
                      lib.gla_pages_fork, lib.gla_pages_free, lib.gla_pages_compact,
                      lib.gla_pages_fork_ex, lib.gla_pages_free_ex, lib.gla_pages_compact_ex):
                f.restype = ctypes.c_int
            lib.hda_fwd_workspace_size.argtypes = [hs, opt]
            lib.hda_bwd_workspace_size.argtypes = [hs, opt]
            lib.gla_group_norm_workspace_size.argtypes = [ns, ctypes.c_int]
            lib.gla_pages_workspace_size.argtypes = [i64, i64, i64, i64]
            for f in (lib.hda_fwd_workspace_size, lib.hda_bwd_workspace_size,
                      lib.gla_group_norm_workspace_size, lib.gla_pages_workspace_size):
                f.restype = ctypes.c_size_t
            cs, ss, qs = ctypes.POINTER(_ConvShape), ctypes.POINTER(_SsmShape), ctypes.POINTER(_QkShape)
            lib.gla_conv_fwd.argtypes = [vp] * 6 + [cs, vp]
            lib.gla_conv_bwd.argtypes = [vp] * 10 + [cs] + ws + [vp]
            lib.gla_conv_step.argtypes = [vp] * 6 + [i64, cs, vp]
            lib.ssm_fwd.argtypes = [vp] * 11 + [ss, opt, vp]
            lib.ssm_bwd.argtypes = [vp] * 20 + [ss, opt, vp]
            lib.ssm_step.argtypes = [vp] * 11 + [i64, ss, vp]
            lib.gla_qk_norm_fwd.argtypes = [vp] * 11 + [qs, vp]
            lib.gla_qk_norm_bwd.argtypes = [vp] * 15 + [qs] + ws + [vp]
            for f in (lib.gla_conv_fwd, lib.gla_conv_bwd, lib.gla_conv_step, lib.ssm_fwd, lib.ssm_bwd,
                      lib.ssm_step, lib.gla_qk_norm_fwd, lib.gla_qk_norm_bwd):
                f.restype = ctypes.c_int
            lib.gla_conv_bwd_workspace_size.argtypes = [cs]
            lib.gla_qk_norm_bwd_workspace_size.argtypes = [qs]
            lib.ssm_fwd_workspace_size.argtypes = [ss, opt]
            lib.ssm_bwd_workspace_size.argtypes = [ss, opt]
            for f in (lib.gla_conv_bwd_workspace_size, lib.gla_qk_norm_bwd_workspace_size,
                      lib.ssm_fwd_workspace_size, lib.ssm_bwd_workspace_size):
                f.restype = ctypes.c_size_t
            _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t):
    """A tensor's address as ctypes takes it for a declared pointer argument (None: NULL)."""
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _launch(f, device, *args):
    """f(*args, stream handle) on torch's current stream, with ``device`` current: switching costs
    as much as a small call, so it is only done when another device is. (The raw handle of the
    stream, without a Stream object around it, for the same reason.)"""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _launch(f, device, *args)
    return f(*args, torch._C._cuda_getCurrentRawStream(device.index))


def _on_stream(stream, f, *args, **kwargs):
    """f with ``stream`` current: outputs allocated while another stream is current may come from
    memory that work still pending there uses."""
    with torch.cuda.stream(stream):
        return f(*args, **kwargs)


def _check(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(workspace, device):
    """(address, bytes) of a caller's workspace, or (None, 0)."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return _addr(workspace), workspace.numel() * workspace.element_size()


def options(path: str = "auto", seq_splits: int = 0, workspace: torch.Tensor | None = None,
            gate: str = "key"):
    opt = _Options()
    opt.path = PATHS[path]
    opt.gate = GATES[gate]
    opt.seq_splits = int(seq_splits)
    opt.workspace = None if workspace is None else workspace.data_ptr()
    opt.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return opt


def workspace_size(B, T, H, Dk=128, Dv=128, io="bf16", path="auto", seq_splits=0) -> int:
    opt = options(path, seq_splits)
    return int(load_library().gla_fwd_workspace_size(B, T, H, Dk, Dv,
                                                      IO_BF16 if io == "bf16" else IO_F32,
                                                      ctypes.byref(opt)))


def path_for(B, T, H, Dk=128, Dv=128, io="bf16", path="auto") -> str | None:
    """Name of the path gla_fwd would run ("exact" / "tc"), or None if unsupported."""
    opt = options(path)
    r = int(load_library().gla_path_for(B, T, H, Dk, Dv, IO_BF16 if io == "bf16" else IO_F32,
                                        ctypes.byref(opt)))
    return {1: "exact", 2: "tc"}.get(r)


def gla_fwd(q, k, v, g, scale: float, h0=None, *, o=None, hT=None, return_state: bool = False,
            path: str = "auto", seq_splits: int = 0, workspace=None, gate: str = "key",
            stream=None):
    """GLA prefill forward through ``gla_fwd_ex``.

    q, k: [B,T,H,Dk]; v: [B,T,H,Dv] (all bf16, or all float32); g: float32 log-gates,
    [B,T,H,Dk] (``gate="key"``) or [B,T,H] (``gate="scalar"``: one gate per token and head);
    h0: [B,H,Dk,Dv] float32 or None. Outputs o (same dtype as q) and, when ``return_state``
    or ``hT`` is given, the float32 final state. Returns (o, hT|None). Asynchronous on
    ``stream`` (default: torch's current stream).
    """
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    _check(q, "q", q.dtype, (B, T, H, Dk), dev)
    _check(k, "k", q.dtype, (B, T, H, Dk), dev)
    _check(v, "v", q.dtype, (B, T, H, Dv), dev)
    _check(g, "g", torch.float32, (B, T, H, Dk) if gate == "key" else (B, T, H), dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (B, T, H, Dv), dev)
    if hT is None and return_state:
        hT = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _check(hT, "hT", torch.float32, (B, H, Dk, Dv), dev)
    _workspace(workspace, dev)
    opt = options(path, seq_splits, workspace, gate)
    io = IO_BF16 if q.dtype == torch.bfloat16 else IO_F32
    with torch.cuda.device(dev):
        rc = lib.gla_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), ctypes.c_float(scale), _ptr(h0),
                            _ptr(o), _ptr(hT), B, T, H, Dk, Dv, io, ctypes.byref(opt),
                            _stream_handle(stream))
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc in (6, 9) else ""
        raise GLAError(rc, "gla_fwd_ex", detail)
    return o, hT


def gla_fwd_noalloc(q, k, v, g, scale: float, h0=None, *, o, hT=None, seq_splits: int = 0,
                    stream=None):
    """GLA prefill forward through ``gla_fwd_noalloc``: bf16 q, k, v, o; the library takes
    its scratch from a fixed array compiled into it and allocates no device memory. The
    caller passes the outputs (``o`` and, optionally, ``hT``) already allocated. Calls that
    overlap on the GPU share that array and race; keep them on one stream. Returns (o, hT).
    """
    lib = load_library()
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    for t, name, shape in ((q, "q", (B, T, H, Dk)), (k, "k", (B, T, H, Dk)),
                           (v, "v", (B, T, H, Dv)), (o, "o", (B, T, H, Dv))):
        _check(t, name, torch.bfloat16, shape, dev)
    _check(g, "g", torch.float32, (B, T, H, Dk), dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, Dk, Dv), dev)
    if hT is not None:
        _check(hT, "hT", torch.float32, (B, H, Dk, Dv), dev)
    with torch.cuda.device(dev):
        rc = lib.gla_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), ctypes.c_float(scale),
                                 _ptr(h0), _ptr(o), _ptr(hT), B, T, H, Dk, Dv, int(seq_splits),
                                 _stream_handle(stream))
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc in (6, 9) else ""
        raise GLAError(rc, "gla_fwd_noalloc", detail)
    return o, hT


def gla_fwd_varlen(q, k, v, g, scale: float, cu_seqlens, h0=None, *, o=None, hT=None,
                   return_state: bool = False, path: str = "auto", gate: str = "key",
                   stream=None):
    """GLA prefill over packed sequences through ``gla_fwd_varlen``.

    q, k: [T,H,Dk]; v: [T,H,Dv] (all bf16, or all float32); g: float32 [T,H,Dk] (or [T,H]
    with ``gate="scalar"``); cu_seqlens: int32 [N+1] on the device (sequence i is tokens
    cu_seqlens[i] .. cu_seqlens[i+1]-1); h0: [N,H,Dk,Dv] float32 or None. Returns (o, hT|None).
    """
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    T, H, Dk = q.shape
    Dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    _check(k, "k", q.dtype, (T, H, Dk), dev)
    _check(v, "v", q.dtype, (T, H, Dv), dev)
    _check(g, "g", torch.float32, (T, H, Dk) if gate == "key" else (T, H), dev)
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (N, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((T, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (T, H, Dv), dev)
    if hT is None and return_state:
        hT = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _check(hT, "hT", torch.float32, (N, H, Dk, Dv), dev)
    opt = options(path, 0, None, gate)
    io = IO_BF16 if q.dtype == torch.bfloat16 else IO_F32
    with torch.cuda.device(dev):
        rc = lib.gla_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(g), ctypes.c_float(scale),
                                _ptr(h0), _ptr(o), _ptr(hT), _ptr(cu_seqlens), N, T, H, Dk, Dv,
                                io, ctypes.byref(opt), _stream_handle(stream))
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc == 6 else ""
        raise GLAError(rc, "gla_fwd_varlen", detail)
    return o, hT


def gla_step(q, k, v, g, scale: float, S, *, o=None, stream=None):
    """One decode step through ``gla_step``: q, k [B,H,Dk]; v [B,H,Dv] (all bf16, or all
    float32); g [B,H,Dk] float32 log-gates; S [B,H,Dk,Dv] float32, updated in place
    (S <- diag(exp(g)) S + k^T v). Returns o = scale q S [B,H,Dv] (same dtype as q)."""
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    _check(k, "k", q.dtype, (B, H, Dk), dev)
    _check(v, "v", q.dtype, (B, H, Dv), dev)
    _check(g, "g", torch.float32, (B, H, Dk), dev)
    _check(S, "S", torch.float32, (B, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (B, H, Dv), dev)
    io = IO_BF16 if q.dtype == torch.bfloat16 else IO_F32
    with torch.cuda.device(dev):
        rc = lib.gla_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), ctypes.c_float(scale), _ptr(S),
                          _ptr(o), B, H, Dk, Dv, io, _stream_handle(stream))
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc == 6 else ""
        raise GLAError(rc, "gla_step", detail)
    return o


def gdn_workspace_size(B: int, T: int, H: int, Dk: int, Dv: int) -> int:
    """Bytes of device workspace ``gdn_fwd`` needs for this shape (0 if unsupported)."""
    return int(load_library().gdn_fwd_workspace_size(B, T, H, Dk, Dv))


def gdn_fwd(q, k, v, g, beta, scale: float, h0=None, *, o=None, hT=None,
            return_state: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """Gated delta rule forward through ``gdn_fwd``.

    q, k: [B,T,H,Dk]; v: [B,T,H,Dv] (all bf16, or all float32); g (log-gates) and beta
    (write strengths): float32 [B,T,H]; h0: [B,H,Dk,Dv] float32 or None. ``workspace``: a
    CUDA tensor of at least ``gdn_workspace_size`` bytes, or None for the library's own.
    Returns (o, hT|None).
    """
    lib = load_library()
    if q.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("q/k/v must be bfloat16 or float32")
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a CUDA device")
    _check(k, "k", q.dtype, (B, T, H, Dk), dev)
    _check(v, "v", q.dtype, (B, T, H, Dv), dev)
    _check(g, "g", torch.float32, (B, T, H), dev)
    _check(beta, "beta", torch.float32, (B, T, H), dev)
    if h0 is not None:
        _check(h0, "h0", torch.float32, (B, H, Dk, Dv), dev)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=dev)
    else:
        _check(o, "o", q.dtype, (B, T, H, Dv), dev)
    if hT is None and return_state:
        hT = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=dev)
    elif hT is not None:
        _check(hT, "hT", torch.float32, (B, H, Dk, Dv), dev)
    ws, ws_bytes = _workspace(workspace, dev)
    io = IO_BF16 if q.dtype == torch.bfloat16 else IO_F32
    with torch.cuda.device(dev):
        rc = lib.gdn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), ctypes.c_float(scale),
                         _ptr(h0), _ptr(o), _ptr(hT), B, T, H, Dk, Dv, io, ws, ws_bytes,
                         _stream_handle(stream))
    if rc != GLA_OK:
        detail = lib.gla_last_error_detail().decode() if rc in (6, 9) else ""
        raise GLAError(rc, "gdn_fwd", detail)
    return o, hT


def launch_counter() -> int:
    """Kernel launches the library has issued in this process."""
    return int(load_library().gla_launch_counter())


def workspace_allocations() -> int:
    """Device allocations the library has made for its per-stream workspaces so far."""
    return int(load_library().gla_workspace_allocations())


def last_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error status."""
    return int(load_library().gla_last_device_status(_stream_handle(stream)))
