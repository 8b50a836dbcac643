"""Python binding of the EFLA GB300 library (libefla_gb300.so, C ABI in include/efla.h).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  Tensors are torch CUDA tensors (torch supplies device memory and
the stream); each call passes ``data_ptr()`` values and the current stream to
the C entry point of the same name.  There is no fallback: if the compiled
library is missing or a call fails, an exception is raised.

Method (gist.science summary of arXiv 2512.12602, "Exact Flow Linear Attention:
Exact Solution from Continuous-Time Dynamics", page es, Metodologia item 3):
    S_t = (I - alpha_t k_t k_t^T) S_{t-1} + alpha_t k_t v_t^T,
    alpha_t = (1 - exp(-beta_t ||k_t||^2)) / ||k_t||^2,      o_t = S_t^T q_t.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "EflaError", "load_library", "library_path", "efla_fwd", "efla_fwd_noalloc", "efla_bwd",
    "efla_step",
    "efla_fwd_workspace_size", "efla_bwd_workspace_size", "efla_get_status",
    "efla_fwd_save", "efla_bwd_saved", "efla_fwd_states_size", "efla_bwd_saved_workspace_size",
    "efla_bwd_plan", "efla_mixer_proj", "MixerShape",
    "efla_gated_fwd", "efla_gated_bwd", "efla_gated_step", "GatedShape", "make_gated_shape",
    "efla_gated_fwd_workspace_size", "efla_gated_bwd_workspace_size",
    "efla_norm_fwd", "efla_norm_bwd", "NormShape",
    "F32", "BF16", "EXACT", "EULER", "AUTO", "SIMT", "TENSOR", "efla_tc_selftest", "efla_wait_selftest",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libefla_gb300.so")
# the same library with -DEFLA_DEBUG: tile-level bounds checks on the tensor-core kernels'
# global writes (EFLA_ERR_BOUNDS from efla_get_status); built beside it by build.py
DEBUG_LIB_PATH = os.path.join(_HERE, "libefla_gb300_debug.so")

F32, BF16 = 0, 1
EXACT, EULER = 0, 1
AUTO, SIMT, TENSOR = 0, 1, 2
_STATUS = {0: "EFLA_OK", 1: "EFLA_ERR_INVALID_ARG", 2: "EFLA_ERR_UNSUPPORTED",
           3: "EFLA_ERR_ALIGNMENT", 4: "EFLA_ERR_WORKSPACE", 5: "EFLA_ERR_CUDA",
           6: "EFLA_ERR_TIMEOUT", 7: "EFLA_ERR_BOUNDS"}


class EflaError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)}: {msg}")


class MixerShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("L", ctypes.c_int), ("D", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int)]


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("L", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("chunk", ctypes.c_int),
                ("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("mode", ctypes.c_int),
                ("path", ctypes.c_int)]


_Strides = ctypes.c_longlong * 3
_GATED_ARRAYS = ("q", "k", "v", "g", "beta", "o", "do", "dq", "dk", "dv")


class GatedShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "H", "Hk", "L", "dk", "dv", "dtype", "out_dtype", "mode", "path",
                                            "packed")] + [(n + "_stride", _Strides) for n in _GATED_ARRAYS]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("D", ctypes.c_int), ("x_stride", ctypes.c_longlong),
                ("y_stride", ctypes.c_longlong), ("dtype", ctypes.c_int), ("weight_dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


_lib = None
_vp = ctypes.c_void_p


def library_path() -> str:
    return _LIB_PATH


def load_library(path: Optional[str] = None):
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it first (python -m exact_flow_recurrence_gb300.build)")
    lib = ctypes.CDLL(p)
    sp = ctypes.POINTER(Shape)
    lib.efla_fwd_workspace_size.restype = ctypes.c_size_t
    lib.efla_fwd_workspace_size.argtypes = [sp]
    lib.efla_bwd_workspace_size.restype = ctypes.c_size_t
    lib.efla_bwd_workspace_size.argtypes = [sp]
    lib.efla_fwd.restype = ctypes.c_int
    lib.efla_fwd.argtypes = [sp] + [_vp] * 8 + [ctypes.c_size_t, _vp]
    lib.efla_bwd.restype = ctypes.c_int
    lib.efla_bwd.argtypes = [sp] + [_vp] * 13 + [ctypes.c_size_t, _vp]
    lib.efla_fwd_states_size.restype = ctypes.c_size_t
    lib.efla_fwd_states_size.argtypes = [sp]
    lib.efla_bwd_saved_workspace_size.restype = ctypes.c_size_t
    lib.efla_bwd_saved_workspace_size.argtypes = [sp]
    lib.efla_bwd_plan.restype = ctypes.c_int
    lib.efla_bwd_plan.argtypes = [sp, ctypes.c_size_t]
    lib.efla_fwd_save.restype = ctypes.c_int
    lib.efla_fwd_save.argtypes = [sp] + [_vp] * 8 + [ctypes.c_size_t, _vp, ctypes.c_size_t, _vp]
    lib.efla_bwd_saved.restype = ctypes.c_int
    lib.efla_bwd_saved.argtypes = [sp] + [_vp] * 5 + [ctypes.c_size_t] + [_vp] * 8 + [ctypes.c_size_t, _vp]
    lib.efla_mixer_proj.restype = ctypes.c_int
    lib.efla_mixer_proj.argtypes = [ctypes.POINTER(MixerShape)] + [_vp] * 7
    lib.efla_fwd_noalloc.restype = ctypes.c_int
    lib.efla_fwd_noalloc.argtypes = [sp] + [_vp] * 8
    lib.efla_step.restype = ctypes.c_int
    lib.efla_step.argtypes = [sp] + [_vp] * 7
    gp = ctypes.POINTER(GatedShape)
    for name in ("efla_gated_fwd_workspace_size", "efla_gated_bwd_workspace_size"):
        getattr(lib, name).restype = ctypes.c_size_t
        getattr(lib, name).argtypes = [gp]
    lib.efla_gated_fwd.restype = ctypes.c_int
    lib.efla_gated_fwd.argtypes = [gp] + [_vp] * 10 + [ctypes.c_size_t, _vp]
    lib.efla_gated_bwd.restype = ctypes.c_int
    lib.efla_gated_bwd.argtypes = [gp] + [_vp] * 16 + [ctypes.c_size_t, _vp]
    lib.efla_gated_step.restype = ctypes.c_int
    lib.efla_gated_step.argtypes = [gp] + [_vp] * 7 + [ctypes.c_int, _vp, _vp]
    np_ = ctypes.POINTER(NormShape)
    lib.efla_norm_fwd.restype = ctypes.c_int
    lib.efla_norm_fwd.argtypes = [np_] + [_vp] * 6
    lib.efla_norm_bwd_workspace_size.restype = ctypes.c_size_t
    lib.efla_norm_bwd_workspace_size.argtypes = [np_]
    lib.efla_norm_bwd.restype = ctypes.c_int
    lib.efla_norm_bwd.argtypes = [np_] + [_vp] * 8 + [ctypes.c_size_t, _vp]
    lib.efla_wait_selftest.restype = ctypes.c_int
    lib.efla_wait_selftest.argtypes = [ctypes.c_int, ctypes.c_int, _vp]
    lib.efla_tc_selftest.restype = ctypes.c_int
    lib.efla_tc_selftest.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int] + [_vp] * 5
    lib.efla_get_status.restype = ctypes.c_int
    lib.efla_get_status.argtypes = [_vp]
    lib.efla_status_string.restype = ctypes.c_char_p
    lib.efla_status_string.argtypes = [ctypes.c_int]
    lib.efla_last_error.restype = ctypes.c_char_p
    lib.efla_last_error.argtypes = []
    if path is None:
        _lib = lib
    return lib


def _check(rc: int, where: str):
    if rc != 0:
        raise EflaError(rc, where, load_library().efla_last_error().decode())


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t} (float32 or bfloat16)")


def _tdt(code: int) -> torch.dtype:
    return torch.bfloat16 if code == BF16 else torch.float32


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _out(t: Optional[torch.Tensor], shape, dtype: torch.dtype, device, name: str) -> torch.Tensor:
    """A caller-supplied output as given (its shape and dtype must be the ones the call
    writes), else a fresh one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t


def make_shape(B, H, L, dk, dv, chunk=64, dtype=torch.bfloat16, out_dtype=None,
               mode: int = EXACT, path: int = AUTO) -> Shape:
    out_dtype = dtype if out_dtype is None else out_dtype
    return Shape(B, H, L, dk, dv, chunk, _dt(dtype), _dt(out_dtype), mode, path)


def efla_fwd_workspace_size(shape: Shape) -> int:
    return load_library().efla_fwd_workspace_size(ctypes.byref(shape))


def efla_bwd_workspace_size(shape: Shape) -> int:
    return load_library().efla_bwd_workspace_size(ctypes.byref(shape))


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    """The caller's workspace as given (the library checks its size), else a fresh one."""
    if ws is not None:
        return ws
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def efla_fwd(q, k, v, beta, S0=None, *, chunk: int = 64, out_dtype=None, mode: int = EXACT,
             o=None, S_final=None, workspace=None, want_state: bool = True, stream=None,
             path: int = AUTO):
    """Chunked EFLA forward.  q,k [B,H,L,dk]; v [B,H,L,dv]; beta [B,H,L] fp32; S0 [B,H,dk,dv] fp32.

    Returns (o [B,H,L,dv], S_final [B,H,dk,dv] fp32 or None)."""
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, L, dk, dv, chunk, q.dtype, out_dtype, mode, path)
    o = _out(o, (B, H, L, dv), _tdt(shape.out_dtype), q.device, "o")
    if S_final is not None or want_state:
        S_final = _out(S_final, (B, H, dk, dv), torch.float32, q.device, "S_final")
    ws = _workspace(efla_fwd_workspace_size(shape), q.device, workspace)
    rc = load_library().efla_fwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                 _ptr(S0), _ptr(o), _ptr(S_final), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "efla_fwd")
    return o, S_final


def efla_fwd_states_size(shape: Shape) -> int:
    return load_library().efla_fwd_states_size(ctypes.byref(shape))


def efla_bwd_saved_workspace_size(shape: Shape) -> int:
    return load_library().efla_bwd_saved_workspace_size(ctypes.byref(shape))


def efla_bwd_plan(shape: Shape, free_bytes: int) -> int:
    """1: record the forward's chunk states (efla_fwd_save + efla_bwd_saved); 0: recompute
    them (efla_fwd + efla_bwd); -1: neither fits in free_bytes."""
    return load_library().efla_bwd_plan(ctypes.byref(shape), free_bytes)


def efla_fwd_save(q, k, v, beta, S0=None, *, chunk: int = 64, out_dtype=None, mode: int = EXACT,
                  o=None, S_final=None, states=None, workspace=None, want_state: bool = True,
                  stream=None, path: int = AUTO):
    """efla_fwd that also records every chunk's entering state and corrected values for
    efla_bwd_saved.  Returns (o, S_final or None, states) with states a flat fp32 tensor
    of efla_fwd_states_size bytes."""
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, L, dk, dv, chunk, q.dtype, out_dtype, mode, path)
    o = _out(o, (B, H, L, dv), _tdt(shape.out_dtype), q.device, "o")
    if S_final is not None or want_state:
        S_final = _out(S_final, (B, H, dk, dv), torch.float32, q.device, "S_final")
    nrec = efla_fwd_states_size(shape)
    if states is None:
        states = torch.empty(max(nrec // 4, 4), dtype=torch.float32, device=q.device)
    ws = _workspace(efla_fwd_workspace_size(shape), q.device, workspace)
    rc = load_library().efla_fwd_save(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                      _ptr(S0), _ptr(o), _ptr(S_final), _ptr(states),
                                      states.numel() * states.element_size(), _ptr(ws),
                                      ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "efla_fwd_save")
    return o, S_final, states


def efla_bwd_saved(q, k, v, beta, dO, states, dS_final=None, *, chunk: int = 64, out_dtype=None,
                   mode: int = EXACT, want_dS0: bool = True, workspace=None, stream=None,
                   path: int = AUTO):
    """efla_bwd from the record of efla_fwd_save (same shape, inputs and mode).
    Returns (dq, dk, dv, dbeta, dS0 or None)."""
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, L, dk, dv, chunk, q.dtype, out_dtype, mode, path)
    odt = _tdt(shape.out_dtype)
    dq = torch.empty((B, H, L, dk), dtype=odt, device=q.device)
    dkk = torch.empty((B, H, L, dk), dtype=odt, device=q.device)
    dvv = torch.empty((B, H, L, dv), dtype=odt, device=q.device)
    db = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    dS0 = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_dS0 else None
    ws = _workspace(efla_bwd_saved_workspace_size(shape), q.device, workspace)
    rc = load_library().efla_bwd_saved(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                       _ptr(states), states.numel() * states.element_size(), _ptr(dO),
                                       _ptr(dS_final), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(db),
                                       _ptr(dS0), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream))
    _check(rc, "efla_bwd_saved")
    return dq, dkk, dvv, db, dS0


def efla_mixer_proj(x, w, H: int, *, dk: int = 128, q=None, k=None, v=None, beta=None, stream=None):
    """The token mixer's input projections: x [B, L, D] bf16, w [3 H dk + H, D] bf16 ->
    q = (x Wq^T)/sqrt(dk), k, v [B, H, L, dk] bf16 and beta = sigmoid(x Wb^T) [B, H, L] fp32."""
    B, L, D = x.shape
    shape = MixerShape(B, L, D, H, dk)
    q = _out(q, (B, H, L, dk), torch.bfloat16, x.device, "q")
    k = _out(k, (B, H, L, dk), torch.bfloat16, x.device, "k")
    v = _out(v, (B, H, L, dk), torch.bfloat16, x.device, "v")
    beta = _out(beta, (B, H, L), torch.float32, x.device, "beta")
    rc = load_library().efla_mixer_proj(ctypes.byref(shape), _ptr(x), _ptr(w), _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(beta), _stream(stream))
    _check(rc, "efla_mixer_proj")
    return q, k, v, beta


def efla_fwd_noalloc(q, k, v, beta, S0=None, *, chunk: int = 64, out_dtype=None,
                     mode: int = EXACT, o=None, S_final=None, want_state: bool = True,
                     stream=None, path: int = AUTO):
    """efla_fwd for callers that cannot allocate device memory: the scratch is the
    library's own device array (EFLA_NOALLOC_SCRATCH_BYTES), so no workspace is passed.
    Outputs (o, S_final) are still the caller's; pass them in to avoid any allocation here."""
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, L, dk, dv, chunk, q.dtype, out_dtype, mode, path)
    o = _out(o, (B, H, L, dv), _tdt(shape.out_dtype), q.device, "o")
    if S_final is not None or want_state:
        S_final = _out(S_final, (B, H, dk, dv), torch.float32, q.device, "S_final")
    rc = load_library().efla_fwd_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v),
                                         _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_final),
                                         _stream(stream))
    _check(rc, "efla_fwd_noalloc")
    return o, S_final


def efla_bwd(q, k, v, beta, dO, S0=None, dS_final=None, *, chunk: int = 64, out_dtype=None,
             mode: int = EXACT, want_dS0: bool = True, workspace=None, stream=None,
             path: int = AUTO):
    """Backward of efla_fwd.  Returns (dq, dk, dv, dbeta, dS0 or None).
    path=SIMT keeps every product in fp32 on the CUDA cores."""
    B, H, L, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, L, dk, dv, chunk, q.dtype, out_dtype, mode, path)
    odt = _tdt(shape.out_dtype)
    dq = torch.empty((B, H, L, dk), dtype=odt, device=q.device)
    dkk = torch.empty((B, H, L, dk), dtype=odt, device=q.device)
    dvv = torch.empty((B, H, L, dv), dtype=odt, device=q.device)
    db = torch.empty((B, H, L), dtype=torch.float32, device=q.device)
    dS0 = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device) if want_dS0 else None
    ws = _workspace(efla_bwd_workspace_size(shape), q.device, workspace)
    rc = load_library().efla_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                 _ptr(S0), _ptr(dO), _ptr(dS_final), _ptr(dq), _ptr(dkk),
                                 _ptr(dvv), _ptr(db), _ptr(dS0), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "efla_bwd")
    return dq, dkk, dvv, db, dS0


def efla_step(q, k, v, beta, S, *, out_dtype=None, mode: int = EXACT, o=None, stream=None):
    """One decode step, S [B,H,dk,dv] fp32 updated in place.  q,k [B,H,dk]; v [B,H,dv]; beta [B,H].

    Returns o [B,H,dv]."""
    B, H, dk = k.shape
    dv = v.shape[-1]
    shape = make_shape(B, H, 1, dk, dv, 1, q.dtype, out_dtype, mode)
    o = _out(o, (B, H, dv), _tdt(shape.out_dtype), q.device, "o")
    rc = load_library().efla_step(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                  _ptr(S), _ptr(o), _stream(stream))
    _check(rc, "efla_step")
    return o


# ------------------------------------------------------------------ gated delta rule
# A call's geometry (sizes, strides, types, mode) is checked and put into the C struct once, and kept
# by its values; what a call still checks is that its tensors have that geometry and lie on one device.
_plans: dict = {}


def _plan(key, make):
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 4096:
            _plans.clear()
        p = _plans[key] = make()
    return p


def _away(t: torch.Tensor, stream) -> bool:
    """Whether the call has to go to another stream, or to another device than the current one."""
    return stream is not None or (t.is_cuda and t.get_device() != torch.cuda.current_device())


def _elsewhere(t: torch.Tensor, stream, fn, *args, **kw):
    """The call on t's device, where its kernels, their attributes and its stream belong, and on `stream`
    if there is one: its fresh outputs and workspace come from that stream's memory pool, where its
    earlier work, and nothing else's, may still be using them."""
    if not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kw)
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=t.device)
        if s.device != t.device:
            raise ValueError(f"stream: expected one of {t.device}, got one of {s.device}")
        with torch.cuda.stream(s):
            return fn(*args, **kw)


def _current(t: torch.Tensor) -> int:
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ws(nbytes: int, t: torch.Tensor, ws: Optional[torch.Tensor]) -> torch.Tensor:
    """The caller's workspace as given (the library checks its size), else a fresh one beside t."""
    if ws is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=t.device)
    _at(ws, "workspace", t.get_device())
    return ws


def _at(t: torch.Tensor, name: str, dev: int):
    if not t.is_cuda:
        raise ValueError(f"{name}: tensors must be CUDA tensors")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got {t.device}")


def _is(t: Optional[torch.Tensor], name: str, dev: int, shape, dtype, contiguous: bool = False):
    """Pointer of a tensor that has to lie on CUDA device `dev` and have this shape and type (None stays None)."""
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != dev:
        _at(t, name, dev)
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _rows_strides(name: str, shape, stride, packed: bool):
    """{batch, head, token} strides of [B,H,L,d] (packed: [H,T,d]), d contiguous."""
    if shape[-1] > 1 and 0 not in shape and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (0,) + tuple(stride[:-1]) if packed else tuple(stride[:-1])


def make_gated_shape(B, H, Hk, L, dk, dv, dtype=torch.bfloat16, out_dtype=None, mode: int = EULER,
                     path: int = AUTO, packed: bool = False, strides=None) -> GatedShape:
    """strides: {array name: (batch, head, token)} in elements; arrays not named: dense [B,H,L,d]
    (packed: [H,L,d])."""
    out_dtype = dtype if out_dtype is None else out_dtype
    s = GatedShape(B, H, Hk, L, dk, dv, _dt(dtype), _dt(out_dtype), mode, path, int(packed))
    for n in _GATED_ARRAYS:
        heads = Hk if n in ("q", "k", "dq", "dk") else H
        d = 1 if n in ("g", "beta") else dk if n in ("q", "k", "dq", "dk") else dv
        st = (strides or {}).get(n)
        setattr(s, n + "_stride", _Strides(*(st if st is not None else (0 if packed else heads * L * d, L * d, d))))
    return s


def efla_gated_fwd_workspace_size(shape: GatedShape) -> int:
    return load_library().efla_gated_fwd_workspace_size(ctypes.byref(shape))


def efla_gated_bwd_workspace_size(shape: GatedShape) -> int:
    return load_library().efla_gated_bwd_workspace_size(ctypes.byref(shape))


class _GatedPlan:
    """Shapes of a gated call's tensors, its C struct and its workspace."""

    def __init__(self, qs, vs, B, packed, dtype, odt, mode, path, strides, bwd):
        if len(vs) != (3 if packed else 4) or len(qs) != len(vs):
            raise ValueError("q, k, v: expected [B,H,L,d], or [H,T,d] with offsets")
        self.q, self.v, self.s = torch.Size(qs), torch.Size(vs), torch.Size(vs[:-1])
        H, L, dv = vs[-3:]
        Hk, dk = qs[-3], qs[-1]
        if qs[-2] != L or qs[:-3] != vs[:-3]:
            raise ValueError(f"q, k: expected {tuple(vs[:-3]) + (Hk, L, dk)}, got {tuple(qs)}")
        self.state = torch.Size((B, H, dk, dv))
        st = {}
        for n, x in strides.items():
            if x is not None:
                shape = self.s if n in ("g", "beta") else self.q if n in ("q", "k", "dq", "dk") else self.v
                if len(x) == len(shape):     # (a tensor of another shape is refused where it is passed)
                    st[n] = ((0,) + tuple(x) if packed else tuple(x)) if n in ("g", "beta") \
                        else _rows_strides(n, shape, x, packed)
        self.shape = make_gated_shape(B, H, Hk, L, dk, dv, dtype, odt, mode, path, packed, st)
        self.ref = ctypes.byref(self.shape)
        self.ws = (efla_gated_bwd_workspace_size if bwd else efla_gated_fwd_workspace_size)(self.shape)


def _batch(v, offsets):
    _at(v, "v", v.get_device())
    if offsets is None:
        return v.shape[0]
    _at(offsets, "offsets", v.get_device())
    if not offsets.is_cuda or offsets.dtype != torch.int32 or offsets.dim() != 1 or offsets.numel() < 1 \
            or not offsets.is_contiguous():
        raise ValueError("offsets: expected a contiguous CUDA int32 tensor [B + 1]")
    return offsets.numel() - 1


def efla_gated_fwd(q, k, v, g, beta, S0=None, *, offsets=None, out_dtype=None, mode: int = EULER, o=None,
                   S_final=None, workspace=None, want_state: bool = True, stream=None, path: int = AUTO):
    """Chunked gated delta rule: S <- e^g S, S <- S + alpha k (v - S^T k)^T, o = S^T q.

    q, k [B,Hk,L,dk], v [B,H,L,dv] (any strides, last dimension contiguous), g (log decay) and beta
    [B,H,L] fp32, S0 [B,H,dk,dv] fp32.  With offsets (int32 [B+1] on the GPU) the sequences are packed
    on one axis of tokens: q, k [Hk,T,dk], v [H,T,dv], g, beta [H,T].
    Returns (o, in v's order of storage, S_final [B,H,dk,dv] fp32 or None)."""
    if _away(v, stream):
        return _elsewhere(v, stream, efla_gated_fwd, q, k, v, g, beta, S0, offsets=offsets, out_dtype=out_dtype, mode=mode, o=o,
                          S_final=S_final, workspace=workspace, want_state=want_state, path=path)
    dt, B, dev = v.dtype, _batch(v, offsets), v.get_device()
    odt = dt if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty_like(v, dtype=odt)
    strides = (q.stride(), k.stride(), v.stride(), g.stride(), beta.stride(), o.stride())
    pl = _plan(("gf", q.shape, v.shape, strides, dt, odt, mode, path, B, offsets is None), lambda: _GatedPlan(
        q.shape, v.shape, B, offsets is not None, dt, odt, mode, path,
        dict(zip(("q", "k", "v", "g", "beta", "o"), strides)), False))
    if S_final is None and want_state:
        S_final = torch.empty(pl.state, dtype=torch.float32, device=v.device)
    ws = _ws(pl.ws, v, workspace)
    f32 = torch.float32
    rc = load_library().efla_gated_fwd(
        pl.ref, None if offsets is None else offsets.data_ptr(), _is(q, "q", dev, pl.q, dt), _is(k, "k", dev, pl.q, dt),
        _is(v, "v", dev, pl.v, dt), _is(g, "g", dev, pl.s, f32), _is(beta, "beta", dev, pl.s, f32),
        _is(S0, "S0", dev, pl.state, f32, True),
        _is(o, "o", dev, pl.v, odt), _is(S_final, "S_final", dev, pl.state, f32, True), _ptr(ws), ws.numel() * ws.element_size(),
        _current(v))
    _check(rc, "efla_gated_fwd")
    return o, S_final


def efla_gated_bwd(q, k, v, g, beta, dO, S0=None, dS_final=None, *, offsets=None, out_dtype=None,
                   mode: int = EULER, dq=None, dk=None, dv=None, want_dS0: bool = True, workspace=None,
                   stream=None, path: int = AUTO):
    """Backward of efla_gated_fwd (same shapes; dO as v).  Returns (dq, dk, dv, dg, dbeta, dS0 or None):
    dq, dk, dv in the order of storage of q, k, v, or into the tensors given (which may be slices of one
    buffer); dg, dbeta fp32, dense."""
    if _away(v, stream):
        return _elsewhere(v, stream, efla_gated_bwd, q, k, v, g, beta, dO, S0, dS_final, offsets=offsets, out_dtype=out_dtype,
                          mode=mode, dq=dq, dk=dk, dv=dv, want_dS0=want_dS0, workspace=workspace, path=path)
    dt, B, f32, dev = v.dtype, _batch(v, offsets), torch.float32, v.get_device()
    odt = dt if out_dtype is None else out_dtype
    dq = torch.empty_like(q, dtype=odt) if dq is None else dq
    dk = torch.empty_like(k, dtype=odt) if dk is None else dk
    dv = torch.empty_like(v, dtype=odt) if dv is None else dv
    strides = (q.stride(), k.stride(), v.stride(), g.stride(), beta.stride(), dO.stride(), dq.stride(), dk.stride(),
               dv.stride())
    pl = _plan(("gb", q.shape, v.shape, strides, dt, odt, mode, path, B, offsets is None), lambda: _GatedPlan(
        q.shape, v.shape, B, offsets is not None, dt, odt, mode, path,
        dict(zip(("q", "k", "v", "g", "beta", "do", "dq", "dk", "dv"), strides)), True))
    dg = torch.empty(pl.s, dtype=f32, device=v.device)
    db = torch.empty(pl.s, dtype=f32, device=v.device)
    dS0 = torch.empty(pl.state, dtype=f32, device=v.device) if want_dS0 else None
    ws = _ws(pl.ws, v, workspace)
    rc = load_library().efla_gated_bwd(
        pl.ref, None if offsets is None else offsets.data_ptr(), _is(q, "q", dev, pl.q, dt), _is(k, "k", dev, pl.q, dt),
        _is(v, "v", dev, pl.v, dt), _is(g, "g", dev, pl.s, f32), _is(beta, "beta", dev, pl.s, f32),
        _is(S0, "S0", dev, pl.state, f32, True),
        _is(dO, "dO", dev, pl.v, dt), _is(dS_final, "dS_final", dev, pl.state, f32, True), _is(dq, "dq", dev, pl.q, odt),
        _is(dk, "dk", dev, pl.q, odt), _is(dv, "dv", dev, pl.v, odt), dg.data_ptr(), db.data_ptr(), _ptr(dS0), _ptr(ws),
        ws.numel() * ws.element_size(), _current(v))
    _check(rc, "efla_gated_bwd")
    return dq, dk, dv, dg, db, dS0


class _StepPlan:
    def __init__(self, qs, vs, S, dtype, odt, mode, strides):
        if len(vs) != 3 or len(qs) != 3 or len(S) != 4:
            raise ValueError("expected q, k [B,Hk,dk], v [B,H,dv], S [n,H,dk,dv]")
        (B, H, dv), (Hk, dk) = vs, qs[1:]
        self.q, self.v, self.s, self.b = torch.Size((B, Hk, dk)), vs, vs[:2], vs[:1]
        self.S = torch.Size((S[0], H, dk, dv))
        st = {}
        for n, x in strides.items():
            if len(x) == 3 and (dk if n in ("q", "k") else dv) > 1 and B * H * Hk and x[2] != 1:
                raise ValueError(f"{n}: the last dimension must be contiguous")
            st[n] = (tuple(x) + (0, 0))[:2] + (0,)
        self.shape = make_gated_shape(B, H, Hk, 1, dk, dv, dtype, odt, mode, AUTO, False, st)
        self.ref = ctypes.byref(self.shape)


def efla_gated_step(q, k, v, g, beta, S, *, slots=None, out_dtype=None, mode: int = EULER, o=None, stream=None):
    """One token of the gated delta rule on a cache of states S [n,H,dk,dv] fp32, updated in place.

    q, k [B,Hk,dk], v [B,H,dv] (any strides, last dimension contiguous), g, beta [B,H] fp32.  slots (int32
    [B] on the GPU): each sequence's place in the cache (outside [0, n): skipped, o = 0); None: place b.
    Returns o [B,H,dv]."""
    if _away(v, stream):
        return _elsewhere(v, stream, efla_gated_step, q, k, v, g, beta, S, slots=slots, out_dtype=out_dtype, mode=mode, o=o)
    dt, f32, dev = v.dtype, torch.float32, v.get_device()
    odt = dt if out_dtype is None else out_dtype
    if o is None:
        o = torch.empty_like(v, dtype=odt)
    strides = (q.stride(), k.stride(), v.stride(), g.stride(), beta.stride(), o.stride())
    pl = _plan(("gs", q.shape, v.shape, S.shape, strides, dt, odt, mode), lambda: _StepPlan(
        q.shape, v.shape, S.shape, dt, odt, mode, dict(zip(("q", "k", "v", "g", "beta", "o"), strides))))
    rc = load_library().efla_gated_step(
        pl.ref, _is(q, "q", dev, pl.q, dt), _is(k, "k", dev, pl.q, dt), _is(v, "v", dev, pl.v, dt), _is(g, "g", dev, pl.s, f32),
        _is(beta, "beta", dev, pl.s, f32), _is(S, "S", dev, pl.S, f32, True),
        _is(slots, "slots", dev, pl.b, torch.int32, True), pl.S[0], _is(o, "o", dev, pl.v, odt), _current(v))
    _check(rc, "efla_gated_step")
    return o


# ------------------------------------------------------------------ layer norm
def _row_stride(name: str, shape, stride) -> int:
    """The one stride that the rows of [..., D] lie apart (D if there is one row, or none)."""
    if len(shape) < 1 or (shape[-1] > 1 and 0 not in shape and stride[-1] != 1):
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if 0 in shape:
        return shape[-1]
    step = span = None
    for n, s in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n == 1:
            continue
        if step is None:
            step, span = s, n * s
        elif s == span:
            span = n * s
        else:
            raise ValueError(f"{name}: its rows must lie one stride apart")
    return shape[-1] if step is None else step


class _NormPlan:
    def __init__(self, shape, xs, ys, dtype, wdtype, eps, bwd):
        D = shape[-1] if len(shape) else 0
        rows = 1
        for n in shape[:-1]:
            rows *= n
        self.x, self.w, self.stats = shape, torch.Size((D,)), torch.Size(tuple(shape[:-1]) + (2,))
        s = self.shape = NormShape(rows, D, _row_stride("x", shape, xs), _row_stride("dy" if bwd else "y", shape, ys),
                                   _dt(dtype), _dt(wdtype), eps)
        self.ref = ctypes.byref(s)
        self.ws = load_library().efla_norm_bwd_workspace_size(self.ref) if bwd else 0


def efla_norm_fwd(x, weight, bias=None, *, eps: float = 1e-5, y=None, stats=None, stream=None):
    """Layer norm over the last dimension of x [..., D].  weight, bias [D] (fp32 or bf16).

    Returns (y like x, stats [..., 2] fp32: mean and 1/sqrt(var + eps) of each row)."""
    if _away(x, stream):
        return _elsewhere(x, stream, efla_norm_fwd, x, weight, bias, eps=eps, y=y, stats=stats)
    dev = x.get_device()
    if y is None:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    pl = _plan(("nf", x.shape, x.stride(), y.stride(), x.dtype, weight.dtype, eps),
               lambda: _NormPlan(x.shape, x.stride(), y.stride(), x.dtype, weight.dtype, eps, False))
    if stats is None:
        stats = torch.empty(pl.stats, dtype=torch.float32, device=x.device)
    rc = load_library().efla_norm_fwd(
        pl.ref, _is(x, "x", dev, pl.x, x.dtype), _is(weight, "weight", dev, pl.w, weight.dtype, True),
        _is(bias, "bias", dev, pl.w, weight.dtype, True), _is(y, "y", dev, pl.x, x.dtype),
        _is(stats, "stats", dev, pl.stats, torch.float32, True), _current(x))
    _check(rc, "efla_norm_fwd")
    return y, stats


def efla_norm_bwd(x, weight, dy, stats, *, want_bias: bool = True, workspace=None, stream=None):
    """Backward of efla_norm_fwd.  Returns (dx dense, dweight, dbias or None), the last two in weight's type."""
    if _away(x, stream):
        return _elsewhere(x, stream, efla_norm_bwd, x, weight, dy, stats, want_bias=want_bias, workspace=workspace)
    dt, wdt, dev = x.dtype, weight.dtype, x.get_device()
    pl = _plan(("nb", x.shape, x.stride(), dy.stride(), dt, wdt),
               lambda: _NormPlan(x.shape, x.stride(), dy.stride(), dt, wdt, 0.0, True))
    dx = torch.empty(pl.x, dtype=dt, device=x.device)
    dw = torch.empty(pl.w, dtype=wdt, device=x.device)
    db = torch.empty(pl.w, dtype=wdt, device=x.device) if want_bias else None
    ws = _ws(pl.ws, x, workspace)
    rc = load_library().efla_norm_bwd(
        pl.ref, _is(x, "x", dev, pl.x, dt), _is(weight, "weight", dev, pl.w, wdt, True), _is(dy, "dy", dev, pl.x, dt),
        _is(stats, "stats", dev, pl.stats, torch.float32, True), dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ws),
        ws.numel() * ws.element_size(), _current(x))
    _check(rc, "efla_norm_bwd")
    return dx, dw, db


def efla_tc_selftest(A, B, C, a_mn_major=False, b_mn_major=False, a_in_tmem=False, stream=None):
    """Diagnostic tile product on tcgen05: returns C + A B^T (A [128,K], B [N,K] fp16; C fp32).

    With a_mn_major / b_mn_major the operand is staged in the MN-major layout (the
    library is handed its transpose); with a_in_tmem, A is read from tensor memory."""
    N, K = B.shape
    D = torch.empty((128, N), dtype=torch.float32, device=A.device)
    a = A.t().contiguous() if a_mn_major else A
    b = B.t().contiguous() if b_mn_major else B
    flags = (1 if a_mn_major else 0) | (2 if b_mn_major else 0) | (4 if a_in_tmem else 0)
    rc = load_library().efla_tc_selftest(N, K, flags, _ptr(a), _ptr(b), _ptr(C), _ptr(D),
                                         _stream(stream))
    _check(rc, "efla_tc_selftest")
    return D


def efla_wait_selftest(kind, limit=4096, stream=None):
    """Diagnostic: a bounded device-side wait that must time out (kind 0: an mbarrier,
    kind 1: a global flag); the next efla_get_status raises EFLA_ERR_TIMEOUT."""
    _check(load_library().efla_wait_selftest(int(kind), int(limit), _stream(stream)), "efla_wait_selftest")


def efla_get_status(stream=None):
    """Synchronise the stream and raise on any asynchronous kernel error."""
    _check(load_library().efla_get_status(_stream(stream)), "efla_get_status")
