"""Thin ctypes binding over libpoetx (include/poetx.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  PyTorch supplies device memory (its caching allocator) and the
current HIP stream.  A nonzero status from the library raises ``PoetxError``.
If the shared library is missing this module raises at import: there is no
fallback path.

Python names mirror the C entry points:
    poetx_merge_perm, poetx_cnp, poetx_forward, poetx_backward,
    poetx_layernorm_forward / _backward, poetx_linear_forward / _backward,
    poetx_xent_forward / _backward (the operators around the layer),
    poetx_glu_forward / _backward, poetx_policy_loss, poetx_grad_norm, poetx_grad_clip
    (those of a fine-tuning step)
plus ``Layer`` (the poetx_layer descriptor) and the measurement hooks.
"""

from __future__ import annotations

import ctypes
import functools
import os
import threading
import weakref
from dataclasses import dataclass
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpoetx.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(
        f"{_LIB_PATH} is missing: build it with `python -m orthogonal_reparameterized_amd.build`")
_lib = ctypes.CDLL(_LIB_PATH)

POETX_OK, POETX_ERR_INVALID_ARG, POETX_ERR_SHAPE = 0, -1, -2
POETX_ERR_UNSUPPORTED, POETX_ERR_WORKSPACE, POETX_ERR_HIP = -3, -4, -5
POETX_F32, POETX_BF16, POETX_I8 = 0, 1, 2
POETX_FAST, POETX_MEM = 0, 1
POETX_CNP_FWD, POETX_CNP_BWD = 0, 1
POETX_ACT_NONE, POETX_ACT_RELU, POETX_ACT_GELU, POETX_ACT_GELU_TANH, POETX_ACT_SILU = 0, 1, 2, 3, 4

POETX_REDUCE_TOKEN, POETX_REDUCE_SEQUENCE, POETX_REDUCE_SUM = 0, 1, 2

_vp, _i64, _i32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


class PoetxLayerC(ctypes.Structure):
    _fields_ = [
        ("d_in", _i64), ("d_out", _i64), ("b", _i64),
        ("act_dtype", _i32), ("w_dtype", _i32), ("g_dtype", _i32), ("variant", _i32),
        ("w_merged", _vp), ("w_merged_t", _vp), ("w_scale", _vp), ("perm_in", _vp), ("perm_out", _vp),
        ("theta_r", _vp), ("theta_p", _vp), ("g_r", _vp), ("g_p", _vp), ("theta_dtype", _i32),
        ("q_r", _vp), ("q_p", _vp),
    ]


class PoetxAdamC(ctypes.Structure):
    _fields_ = [
        ("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
        ("gamma", ctypes.c_float), ("step", _i64),
        ("m_r", _vp), ("v_r", _vp), ("m_p", _vp), ("v_p", _vp), ("theta_r_out", _vp), ("theta_p_out", _vp),
    ]


class PoetxPolicyC(ctypes.Structure):
    _fields_ = [
        ("clip_low", ctypes.c_double), ("clip_high", ctypes.c_double), ("beta", ctypes.c_double),
        ("scale", ctypes.c_double), ("reduce", _i32), ("adv_per_token", _i32),
    ]


class PoetxGradC(ctypes.Structure):
    _fields_ = [("g", _vp), ("out", _vp), ("n", _i64), ("dtype", _i32)]


_lib.poetx_merge_perm.argtypes = [_vp, _vp, _i32, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.poetx_cnp.argtypes = [_i32, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp,
                           ctypes.POINTER(_sz), _vp]
_lib.poetx_forward.argtypes = [ctypes.POINTER(PoetxLayerC), _i64, _vp, _vp, _vp, _vp, _vp,
                               ctypes.POINTER(_sz), _vp]
_lib.poetx_backward.argtypes = [ctypes.POINTER(PoetxLayerC), _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                _vp, _vp, _vp, _vp, ctypes.POINTER(_sz), _vp]
_lib.poetx_cnp_noalloc.argtypes = [_i32, _i64, _i64, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp]
_lib.poetx_backward_adam.argtypes = [ctypes.POINTER(PoetxLayerC), _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     ctypes.POINTER(PoetxAdamC), _vp, ctypes.POINTER(_sz), _vp]
_lib.poetx_fold.argtypes = [ctypes.POINTER(PoetxLayerC), _vp, _vp, ctypes.POINTER(_sz), _vp]
_lib.poetx_adam_step.argtypes = [_i64, _vp, _i32, _vp, _vp, _vp, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                 ctypes.c_float, _i64, ctypes.c_float, _vp]
_szp = ctypes.POINTER(_sz)
_lib.poetx_layernorm_forward.argtypes = [_i64, _i64, _i32, _vp, _vp, _vp, _i32, ctypes.c_float, _vp, _vp, _vp, _vp]
_lib.poetx_layernorm_backward.argtypes = [_i64, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                          _szp, _vp]
_lib.poetx_linear_forward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _szp,
                                      _vp]
_lib.poetx_linear_backward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_xent_forward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_xent_backward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_glu_forward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_glu_backward.argtypes = [_i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp,
                                    _szp, _vp]
_lib.poetx_policy_loss.argtypes = [_i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_grad_plan.argtypes = [_i64, _vp, _vp, _szp, _vp]
_lib.poetx_grad_norm.argtypes = [_i64, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_grad_clip.argtypes = [_i64, _vp, ctypes.c_float, _vp, _vp, _vp, _vp, _szp, _vp]
_lib.poetx_status_string.argtypes = [ctypes.c_int]
_lib.poetx_status_string.restype = ctypes.c_char_p
_lib.poetx_version.restype = ctypes.c_char_p
_lib.poetx_prof_enable.argtypes = [_i32]
_lib.poetx_prof_read.argtypes = [ctypes.c_char_p, _sz]
_lib.poetx_prof_only.argtypes = [ctypes.c_char_p]
for _f in ("poetx_merge_perm", "poetx_cnp", "poetx_cnp_noalloc", "poetx_forward", "poetx_backward", "poetx_backward_adam", "poetx_fold",
           "poetx_adam_step", "poetx_layernorm_forward", "poetx_layernorm_backward", "poetx_linear_forward",
           "poetx_linear_backward", "poetx_xent_forward", "poetx_xent_backward", "poetx_glu_forward",
           "poetx_glu_backward", "poetx_policy_loss", "poetx_grad_plan", "poetx_grad_norm", "poetx_grad_clip",
           "poetx_prof_enable", "poetx_prof_only", "poetx_prof_read"):
    getattr(_lib, _f).restype = ctypes.c_int

EXPORTED = ("poetx_merge_perm", "poetx_cnp", "poetx_cnp_noalloc", "poetx_forward", "poetx_backward", "poetx_backward_adam", "poetx_fold",
            "poetx_adam_step", "poetx_layernorm_forward", "poetx_layernorm_backward", "poetx_linear_forward",
            "poetx_linear_backward", "poetx_xent_forward", "poetx_xent_backward", "poetx_glu_forward",
            "poetx_glu_backward", "poetx_policy_loss", "poetx_grad_plan", "poetx_grad_norm", "poetx_grad_clip",
            "poetx_status_string", "poetx_version", "poetx_prof_enable", "poetx_prof_only", "poetx_prof_read")


class PoetxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.poetx_status_string(status).decode()} ({status})")


def _check(st: int, where: str):
    if st != POETX_OK:
        raise PoetxError(st, where)


def library_path() -> str:
    return _LIB_PATH


def version() -> str:
    return _lib.poetx_version().decode()


_DT = {torch.float32: POETX_F32, torch.bfloat16: POETX_BF16, torch.int8: POETX_I8}


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _ptr(t: Optional[torch.Tensor], align: int = 16):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    if t.data_ptr() % align:
        raise ValueError(f"tensor must be {align}-byte aligned")
    return ctypes.c_void_p(t.data_ptr())


# the current HIP stream of a device by its index, without building a torch Stream object (2 us)
# where torch has that internal function
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda idx: torch.cuda.current_stream(idx).cuda_stream)


def _stream(dev: torch.device):
    return ctypes.c_void_p(_raw_stream(dev.index if dev.index is not None else torch.cuda.current_device()))


# Scratch tensors keyed by (device, stream): each is allocated while its stream is the
# current one and only ever used by calls on that stream, so the caching allocator's
# stream ordering makes both the reuse between calls and the release of an outgrown
# buffer safe.  Layers driven on different streams get different workspaces.  A call that is
# being captured into a graph takes a workspace of its own from the graph's memory pool: it
# lives as long as the graph, and no eager call or other graph shares it.  Each thread has its
# own workspaces: a call launches several kernels, and another thread's may come between them
# on the same stream.  They go with their thread, or all at once by release_workspace().
class _WsCache(dict):
    __slots__ = ("__weakref__",)
    __hash__, __eq__ = object.__hash__, object.__eq__  # an element of a WeakSet by identity


_ws_all: weakref.WeakSet = weakref.WeakSet()
_ws_lock = threading.Lock()


class _WsLocal(threading.local):
    def __init__(self):  # runs once in every thread that reaches for its workspaces
        self.cache = _WsCache()
        with _ws_lock:
            _ws_all.add(self.cache)


_ws_local = _WsLocal()
_capturing = torch.cuda.is_current_stream_capturing


def _workspace(dev: torch.device, nbytes: int) -> torch.Tensor:
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    if _capturing():
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{idx}")
    key = (idx, _raw_stream(idx))
    cache = _ws_local.cache
    t = cache.get(key)
    if t is None or t.numel() < nbytes:
        with torch.cuda.device(idx):
            t = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=f"cuda:{idx}")
        cache[key] = t
    return t


def release_workspace():
    """Drop every cached workspace, those of other threads as well.  (A call that is under way in
    another thread holds its own until its kernels are launched; the allocator hands the memory
    on in the order of the stream they run on.)"""
    with _ws_lock:
        caches = list(_ws_all)
    for cache in caches:
        cache.clear()


# --------------------------------------------------------------------------
def poetx_merge_perm(w: torch.Tensor, perm_out=None, perm_in=None, w_scale=None,
                     out: Optional[torch.Tensor] = None, out_scale: Optional[torch.Tensor] = None,
                     out_t: Optional[torch.Tensor] = None):
    """W'[i][k] = W[perm_out[i]][perm_in[k]] (and s'[i] = s[perm_out[i]] for int8).

    If out_t is given it also receives W'^T ([d_in][d_out]).
    """
    d_out, d_in = w.shape
    out = torch.empty_like(w) if out is None else out
    if w.dtype == torch.int8 and out_scale is None:
        out_scale = torch.empty_like(w_scale)
    st = _lib.poetx_merge_perm(_ptr(w), _ptr(w_scale), _dt(w), d_out, d_in, _ptr(perm_out),
                               _ptr(perm_in), _ptr(out), _ptr(out_scale) if w.dtype == torch.int8 else None,
                               _ptr(out_t), _stream(w.device))
    _check(st, "poetx_merge_perm")
    return out, (out_scale if w.dtype == torch.int8 else None)


def _need(t: Optional[torch.Tensor], name: str, numel: int, dtypes) -> None:
    """A buffer the library reads or writes through a raw pointer: contiguous, of one of the
    expected dtypes and with exactly the elements the call touches."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def qsave_like(theta: torch.Tensor, b: int) -> torch.Tensor:
    """A buffer for poetx_cnp's qsave (n * b * b * 4 bytes, 16-byte aligned)."""
    return torch.empty((theta.shape[0], b, b), dtype=torch.float32, device=theta.device)


def poetx_cnp(direction: int, theta: torch.Tensor, b: int, *, g: Optional[torch.Tensor] = None,
              g_dtype: torch.dtype = torch.bfloat16, dg: Optional[torch.Tensor] = None,
              dtheta: Optional[torch.Tensor] = None, qsave: Optional[torch.Tensor] = None):
    """FWD: returns G [n][b][b] in g_dtype; BWD: returns dtheta [n][b(b-1)/2] from dg.
    qsave (optional, from qsave_like): FWD fills it, BWD on the same theta reads Q from it."""
    n = theta.shape[0]
    dev = theta.device
    p = b * (b - 1) // 2
    # the library writes through raw pointers: every buffer's dtype and size is checked here
    _need(theta, "theta", n * p, (torch.float32, torch.bfloat16))
    if direction == POETX_CNP_FWD:
        g = torch.empty((n, b, b), dtype=g_dtype, device=dev) if g is None else g
        _need(g, "g", n * b * b, (torch.float32, torch.bfloat16))
        gdt, dgdt = _dt(g), POETX_F32
    else:
        dtheta = torch.empty(theta.shape, dtype=torch.float32, device=dev) if dtheta is None else dtheta
        _need(dg, "dg", n * b * b, (torch.float32,))
        _need(dtheta, "dtheta", n * p, (torch.float32,))
        gdt, dgdt = POETX_F32, _dt(dg)
    if qsave is not None:
        _need(qsave, "qsave", n * b * b, (torch.float32,))
    tdt = _dt(theta)
    nbytes = _sz(0)
    _check(_lib.poetx_cnp(direction, n, b, None, tdt, None, gdt, None, None, dgdt, None, None,
                          ctypes.byref(nbytes), None), "poetx_cnp(size)")
    ws = _workspace(dev, nbytes.value)
    nb = _sz(ws.numel())
    # poetx_cnp takes element-aligned theta, G and dG (a smaller last block of a side
    # sits at an offset of whole blocks, which need not be a multiple of 16 bytes)
    def ep(t):
        return None if t is None else _ptr(t, t.element_size())
    st = _lib.poetx_cnp(direction, n, b, ep(theta), tdt, ep(g), gdt, _ptr(qsave), ep(dg), dgdt, ep(dtheta),
                        _ptr(ws), ctypes.byref(nb), _stream(dev))
    _check(st, "poetx_cnp")
    return g if direction == POETX_CNP_FWD else dtheta


@dataclass
class Layer:
    """Python view of poetx_layer: the tensors stay owned by the caller."""
    w_merged: torch.Tensor
    theta_r: torch.Tensor
    theta_p: torch.Tensor
    g_r: torch.Tensor
    g_p: torch.Tensor
    b: int
    act_dtype: torch.dtype = torch.bfloat16
    variant: int = POETX_FAST
    w_scale: Optional[torch.Tensor] = None
    perm_in: Optional[torch.Tensor] = None
    perm_out: Optional[torch.Tensor] = None
    w_merged_t: Optional[torch.Tensor] = None
    q_r: Optional[torch.Tensor] = None    # qsave buffers the CNP forward filled (full blocks)
    q_p: Optional[torch.Tensor] = None

    @property
    def d_out(self):
        return self.w_merged.shape[0]

    @property
    def d_in(self):
        return self.w_merged.shape[1]

    def to_c(self) -> PoetxLayerC:
        c = PoetxLayerC()
        c.d_in, c.d_out, c.b = self.d_in, self.d_out, self.b
        c.act_dtype = _DT[self.act_dtype]
        c.w_dtype = _dt(self.w_merged)
        c.g_dtype = _dt(self.g_r)
        c.variant = self.variant
        c.theta_dtype = _dt(self.theta_r)
        for q, d in ((self.q_r, self.d_in), (self.q_p, self.d_out)):
            if q is not None:
                _need(q, "q_r / q_p", (d // self.b) * self.b * self.b, (torch.float32,))
        for name in ("w_merged", "w_merged_t", "w_scale", "perm_in", "perm_out", "theta_r", "theta_p",
                     "g_r", "g_p", "q_r", "q_p"):
            p = _ptr(getattr(self, name))
            setattr(c, name, p.value if p is not None else None)
        return c


def poetx_forward(layer: Layer, x: torch.Tensor, z: Optional[torch.Tensor] = None,
                  saved_b: Optional[torch.Tensor] = None, saved_x: Optional[torch.Tensor] = None):
    """Returns (z, saved_b); saved_b is None for the mem variant.  saved_x (fast variant,
    optional, [N][d_in]) receives the gathered input for poetx_backward."""
    L = layer.to_c()
    n = x.shape[0]
    dev = x.device
    z = torch.empty((n, layer.d_out), dtype=layer.act_dtype, device=dev) if z is None else z
    if layer.variant == POETX_FAST and saved_b is None:
        saved_b = torch.empty((n, layer.d_out), dtype=layer.act_dtype, device=dev)
    if layer.variant == POETX_MEM:
        saved_b = None
    nbytes = _sz(0)
    _check(_lib.poetx_forward(ctypes.byref(L), n, None, None, None, _ptr(saved_x), None, ctypes.byref(nbytes),
                              None), "poetx_forward(size)")
    ws = _workspace(dev, nbytes.value)
    nb = _sz(ws.numel())
    st = _lib.poetx_forward(ctypes.byref(L), n, _ptr(x), _ptr(z), _ptr(saved_b), _ptr(saved_x), _ptr(ws),
                            ctypes.byref(nb), _stream(dev))
    _check(st, "poetx_forward")
    return z, saved_b


def poetx_backward(layer: Layer, x: torch.Tensor, dz: torch.Tensor,
                   saved_b: Optional[torch.Tensor] = None, *, saved_x=None, dx=None, dtheta_r=None,
                   dtheta_p=None, want_dg: bool = False):
    """Returns dict(dx, dtheta_r, dtheta_p[, dg_r, dg_p]).  saved_x: what poetx_forward wrote
    into its saved_x, or None."""
    L = layer.to_c()
    n = x.shape[0]
    dev = x.device
    dx = torch.empty((n, layer.d_in), dtype=layer.act_dtype, device=dev) if dx is None else dx
    dtheta_r = torch.empty(layer.theta_r.shape, dtype=torch.float32, device=dev) if dtheta_r is None else dtheta_r
    dtheta_p = torch.empty(layer.theta_p.shape, dtype=torch.float32, device=dev) if dtheta_p is None else dtheta_p
    _need(dx, "dx", n * layer.d_in, (layer.act_dtype,))
    _need(dtheta_r, "dtheta_r", layer.theta_r.numel(), (torch.float32,))
    _need(dtheta_p, "dtheta_p", layer.theta_p.numel(), (torch.float32,))
    dg_r = dg_p = None
    if want_dg:
        b = layer.b
        if layer.d_in % b or layer.d_out % b:  # flat: full blocks, then the smaller last block
            dg_r = torch.empty((layer.d_in // b) * b * b + (layer.d_in % b) ** 2, dtype=torch.float32, device=dev)
            dg_p = torch.empty((layer.d_out // b) * b * b + (layer.d_out % b) ** 2, dtype=torch.float32,
                               device=dev)
        else:
            dg_r = torch.empty((layer.d_in // b, b, b), dtype=torch.float32, device=dev)
            dg_p = torch.empty((layer.d_out // b, b, b), dtype=torch.float32, device=dev)
    nbytes = _sz(0)
    _check(_lib.poetx_backward(ctypes.byref(L), n, None, None, None, _ptr(saved_x), None, None, None,
                               _ptr(dg_r), _ptr(dg_p), None, ctypes.byref(nbytes), None), "poetx_backward(size)")
    ws = _workspace(dev, nbytes.value)
    nb = _sz(ws.numel())
    st = _lib.poetx_backward(ctypes.byref(L), n, _ptr(x), _ptr(dz), _ptr(saved_b), _ptr(saved_x), _ptr(dx),
                             _ptr(dtheta_r), _ptr(dtheta_p), _ptr(dg_r), _ptr(dg_p), _ptr(ws),
                             ctypes.byref(nb), _stream(dev))
    _check(st, "poetx_backward")
    out = dict(dx=dx, dtheta_r=dtheta_r, dtheta_p=dtheta_p)
    if want_dg:
        out.update(dg_r=dg_r, dg_p=dg_p)
    return out


def poetx_fold(layer: Layer, w_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The layer's effective weight [d_out][d_in] in original coordinates (see poetx.h)."""
    L = layer.to_c()
    dev = layer.w_merged.device
    if w_out is None:
        w_out = torch.empty((layer.d_out, layer.d_in), dtype=layer.w_merged.dtype, device=dev)
    nbytes = _sz(0)
    _check(_lib.poetx_fold(ctypes.byref(L), None, None, ctypes.byref(nbytes), None), "poetx_fold(size)")
    ws = _workspace(dev, nbytes.value)
    nb = _sz(ws.numel())
    _check(_lib.poetx_fold(ctypes.byref(L), _ptr(w_out), _ptr(ws), ctypes.byref(nb), _stream(dev)),
           "poetx_fold")
    return w_out


def poetx_adam_step(theta: torch.Tensor, grad: torch.Tensor, m: torch.Tensor, v: torch.Tensor, *, lr: float,
                    step: int, betas=(0.9, 0.999), eps: float = 1e-8, gamma: float = 1.0):
    """In-place Adam update of packed theta (float32 or bf16) and its float32 state m, v
    from grad = dtheta."""
    _need(theta, "theta", theta.numel(), (torch.float32, torch.bfloat16))
    for t, nm in ((grad, "grad"), (m, "m"), (v, "v")):
        _need(t, nm, theta.numel(), (torch.float32,))
    _check(_lib.poetx_adam_step(theta.numel(), _ptr(theta), _dt(theta), _ptr(grad), _ptr(m), _ptr(v), lr,
                                betas[0], betas[1], eps, step, gamma, _stream(theta.device)), "poetx_adam_step")
    return theta


@dataclass
class AdamState:
    """Adam state of a layer's two packed thetas (float32, theta's layout) and its step."""
    m_r: torch.Tensor
    v_r: torch.Tensor
    m_p: torch.Tensor
    v_p: torch.Tensor
    step: int = 0

    @staticmethod
    def zeros_like(layer: "Layer") -> "AdamState":
        z = [torch.zeros(t.shape, dtype=torch.float32, device=t.device)
             for t in (layer.theta_r, layer.theta_r, layer.theta_p, layer.theta_p)]
        return AdamState(*z)


def poetx_backward_adam(layer: Layer, x: torch.Tensor, dz: torch.Tensor, state: AdamState,
                        saved_b: Optional[torch.Tensor] = None, *, lr: float, betas=(0.9, 0.999),
                        eps: float = 1e-8, gamma: float = 1.0, saved_x=None, dx=None, dtheta_r=None,
                        dtheta_p=None):
    """The backward with one Adam step of layer.theta_r / layer.theta_p (in place) fused into
    the CNP backward's last pass; state.step advances by one.  Returns dict(dx[, dtheta_*])."""
    L = layer.to_c()
    n = x.shape[0]
    dev = x.device
    dx = torch.empty((n, layer.d_in), dtype=layer.act_dtype, device=dev) if dx is None else dx
    _need(dx, "dx", n * layer.d_in, (layer.act_dtype,))
    for t, th, nm in ((state.m_r, layer.theta_r, "m_r"), (state.v_r, layer.theta_r, "v_r"),
                      (state.m_p, layer.theta_p, "m_p"), (state.v_p, layer.theta_p, "v_p")):
        _need(t, nm, th.numel(), (torch.float32,))
    for t, th, nm in ((dtheta_r, layer.theta_r, "dtheta_r"), (dtheta_p, layer.theta_p, "dtheta_p")):
        if t is not None:
            _need(t, nm, th.numel(), (torch.float32,))
    state.step += 1
    opt = PoetxAdamC()
    opt.lr, opt.beta1, opt.beta2, opt.eps, opt.gamma, opt.step = lr, betas[0], betas[1], eps, gamma, state.step
    for name in ("m_r", "v_r", "m_p", "v_p"):
        setattr(opt, name, _ptr(getattr(state, name)).value)
    opt.theta_r_out, opt.theta_p_out = _ptr(layer.theta_r).value, _ptr(layer.theta_p).value
    nbytes = _sz(0)
    _check(_lib.poetx_backward_adam(ctypes.byref(L), n, None, None, None, _ptr(saved_x), None, None, None,
                                    ctypes.byref(opt), None, ctypes.byref(nbytes), None), "poetx_backward_adam(size)")
    ws = _workspace(dev, nbytes.value)
    nb = _sz(ws.numel())
    st = _lib.poetx_backward_adam(ctypes.byref(L), n, _ptr(x), _ptr(dz), _ptr(saved_b), _ptr(saved_x), _ptr(dx),
                                  _ptr(dtheta_r), _ptr(dtheta_p), ctypes.byref(opt), _ptr(ws), ctypes.byref(nb),
                                  _stream(dev))
    _check(st, "poetx_backward_adam")
    out = dict(dx=dx)
    if dtheta_r is not None:
        out.update(dtheta_r=dtheta_r, dtheta_p=dtheta_p)
    return out


# ---------------------------------------------------------------------------
# Operators around the layer: layer norm, dense linear layer, vocabulary cross entropy.
# The last axis of x (h) is the feature axis, the leading axes together are the tokens.
# ---------------------------------------------------------------------------
_FLOATS = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)
_ACTS = {"none": POETX_ACT_NONE, "relu": POETX_ACT_RELU, "gelu": POETX_ACT_GELU, "gelu_tanh": POETX_ACT_GELU_TANH,
         "silu": POETX_ACT_SILU}


def _act(act) -> int:
    if act in _ACTS:
        return _ACTS[act]
    if act in _ACTS.values():
        return act
    raise ValueError(f"act: {act!r}, expected one of {tuple(_ACTS)}")


def _buf(t: Optional[torch.Tensor], name: str, shape, dtypes, dev) -> Optional[int]:
    """The address of an input or output buffer (None for None), once its shape, dtype, layout,
    device and alignment are what the library expects."""
    if t is None:
        return None
    if t.dtype in dtypes and t.shape == shape and t.device == dev and t.is_contiguous():
        p = t.data_ptr()
        if not p & 15:
            return p
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be 16-byte aligned")


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, ref: torch.Tensor):
    """(tensor, address) of an output on ref's device: the caller's, checked, or a new one
    (new_empty and empty_like take half the time of torch.empty with a device)."""
    if t is None:
        t = torch.empty_like(ref) if shape is None else ref.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _buf(t, name, ref.shape if shape is None else shape, (dtype,), ref.device)


def _tokens(t: torch.Tensor, name: str):
    d = t.shape[-1] if t.dim() else 0
    if d < 1:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [..., features]")
    return t.numel() // d, d


@functools.lru_cache(maxsize=1024)
def _ws_query(fn: str, idx: int, args: tuple) -> int:
    """Workspace bytes of a call: what its size query (ws == NULL) answers on device idx, which
    is the current one."""
    nb = _sz(0)
    _check(getattr(_lib, fn)(*args, None, ctypes.byref(nb), None), f"{fn}(size)")
    return nb.value


_SOME = 256  # a non-null pointer for size queries, which look only at which outputs are wanted
_current_device = torch.cuda.current_device
_byref = ctypes.byref


def _run(fn, dev: torch.device, args: tuple, query=None) -> None:
    """The call on dev's current stream, with its workspace when `query` has its size query's
    arguments (or the size itself).  The library launches on the current device, so that is made
    dev's."""
    idx = dev.index
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    if _current_device() != idx:
        with torch.cuda.device(dev):
            return _run(fn, dev, args, query)
    if query is None:
        code = fn(*args, _raw_stream(idx))
    else:
        ws = _workspace(dev, query if type(query) is int else _ws_query(fn.__name__, idx, query))
        code = fn(*args, ws.data_ptr(), _byref(_sz(ws.numel())), _raw_stream(idx))
    if code != POETX_OK:
        _check(code, fn.__name__)


def poetx_layernorm_forward(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                            beta: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                            y: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                            rstd: Optional[torch.Tensor] = None):
    """Layer norm over the last axis.  Returns (y, mean, rstd): mean and rstd float32 [tokens],
    for the backward.  gamma and beta: [d], both float32 or both bf16, each optional."""
    n, d = _tokens(x, "x")
    dev = x.device
    px = _buf(x, "x", x.shape, _FLOATS, dev)
    p = gamma if gamma is not None else beta
    pd = (p.dtype,) if p is not None and p.dtype in _FLOATS else _FLOATS
    pg, pb = _buf(gamma, "gamma", (d,), pd, dev), _buf(beta, "beta", (d,), pd, dev)
    y, py = _out(y, "y", None, x.dtype, x)
    mean, pm = _out(mean, "mean", (n,), torch.float32, x)
    rstd, pr = _out(rstd, "rstd", (n,), torch.float32, x)
    _run(_lib.poetx_layernorm_forward, dev,
         (n, d, _DT[x.dtype], px, pg, pb, _DT[p.dtype] if p is not None else POETX_F32, eps, py, pm, pr))
    return y, mean, rstd


def poetx_layernorm_backward(x: torch.Tensor, dy: torch.Tensor, gamma: Optional[torch.Tensor], mean: torch.Tensor,
                             rstd: torch.Tensor, *, dres: Optional[torch.Tensor] = None,
                             dx: Optional[torch.Tensor] = None, want_params: bool = True):
    """Returns dict(dx[, dgamma, dbeta]); dgamma, dbeta float32 [d].  dres: the gradient that
    reaches x past the norm, added to dx."""
    n, d = _tokens(x, "x")
    dev, shape, dt = x.device, x.shape, (x.dtype,)
    px = _buf(x, "x", shape, _FLOATS, dev)
    ins = (_buf(dy, "dy", shape, dt, dev), _buf(gamma, "gamma", (d,), _FLOATS, dev))
    stats = (_buf(mean, "mean", (n,), _F32, dev), _buf(rstd, "rstd", (n,), _F32, dev),
             _buf(dres, "dres", shape, dt, dev))
    dx, pdx = _out(dx, "dx", None, x.dtype, x)
    pd, code = _DT[gamma.dtype] if gamma is not None else POETX_F32, _DT[x.dtype]
    out, some, params = dict(dx=dx), None, (None, None)
    if want_params:
        out["dgamma"], out["dbeta"] = x.new_empty(d, dtype=torch.float32), x.new_empty(d, dtype=torch.float32)
        some, params = _SOME, (out["dgamma"].data_ptr(), out["dbeta"].data_ptr())
    _run(_lib.poetx_layernorm_backward, dev, (n, d, code, px, *ins, pd, *stats, pdx, *params),
         (n, d, code, None, None, None, pd, None, None, None, None, some, some))
    return out


def poetx_linear_forward(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                         residual: Optional[torch.Tensor] = None, act="none", *, y: Optional[torch.Tensor] = None,
                         save_pre: bool = False):
    """act(x . w^T + bias) + residual.  Returns (y, pre): pre, what the activation took, for
    the backward when save_pre is set, else None.  act: a name ("none", "relu", "gelu",
    "gelu_tanh", "silu") or a POETX_ACT_* code."""
    n, d_in = _tokens(x, "x")
    dev, dt = x.device, (x.dtype,)
    d_out = w.shape[0]
    a = _act(act)
    shape = x.shape[:-1] + (d_out,)
    ins = (_buf(x, "x", x.shape, _FLOATS, dev), _buf(w, "w", (d_out, d_in), dt, dev),
           _buf(bias, "bias", (d_out,), _FLOATS, dev))
    pr = _buf(residual, "residual", shape, dt, dev)
    y, py = _out(y, "y", shape, x.dtype, x)
    pre = torch.empty_like(y) if save_pre else None
    bd, code = _DT[bias.dtype] if bias is not None else POETX_F32, _DT[x.dtype]
    _run(_lib.poetx_linear_forward, dev,
         (n, d_in, d_out, code, *ins, bd, pr, a, py, pre.data_ptr() if save_pre else None),
         (n, d_in, d_out, code, None, None, None, bd, None, a, None, None))
    return y, pre


def poetx_linear_backward(x: Optional[torch.Tensor], w: Optional[torch.Tensor], dy: torch.Tensor,
                          pre: Optional[torch.Tensor] = None, act="none", *, want_dx: bool = True,
                          want_dw: bool = True, want_dbias: bool = True):
    """Returns dict with those of dx, dw (x's dtype) and dbias (float32) that are wanted.  pre:
    what poetx_linear_forward(save_pre=True) returned (not needed for act "none").  x is needed
    for dw, w for dx."""
    n, d_out = _tokens(dy, "dy")
    dev, dt = dy.device, (dy.dtype,)
    a = _act(act)
    if want_dx and w is None or want_dw and x is None:
        raise ValueError("dx needs w, dw needs x")
    if a != POETX_ACT_NONE and pre is None:
        raise ValueError("pre is required for this activation")
    ref = x if x is not None else w
    d_in = ref.shape[-1] if ref is not None else 1
    shape = dy.shape[:-1] + (d_in,)
    pdy = _buf(dy, "dy", dy.shape, _FLOATS, dev)
    ins = (_buf(x, "x", shape, dt, dev), _buf(w, "w", (d_out, d_in), dt, dev), pdy,
           _buf(pre, "pre", dy.shape, dt, dev))
    out, ptrs = {}, []
    for name, want, size, dtype in (("dx", want_dx, shape, dy.dtype), ("dw", want_dw, (d_out, d_in), dy.dtype),
                                    ("dbias", want_dbias, (d_out,), torch.float32)):
        if want:
            out[name] = dy.new_empty(size, dtype=dtype)
        ptrs.append(out[name].data_ptr() if want else None)
    if n == 0 and not (want_dw or want_dbias):
        return out
    code = _DT[dy.dtype]
    _run(_lib.poetx_linear_backward, dev, (n, d_in, d_out, code, *ins, a, *ptrs),
         (n, d_in, d_out, code, None, None, None, None, a, *(None if p is None else _SOME for p in ptrs)))
    return out


def poetx_xent_forward(h: torch.Tensor, w: torch.Tensor, target: torch.Tensor, *,
                       loss: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """Softmax cross entropy of the logits h . w^T, which are not stored.  target: int32, one
    per token; a target outside [0, vocab) marks a token that takes no part (loss 0).  Returns
    (loss, lse), float32, one per token."""
    n, d = _tokens(h, "h")
    dev = h.device
    vocab = w.shape[0]
    lead = h.shape[:-1]
    ins = (_buf(h, "h", h.shape, _FLOATS, dev), _buf(w, "w", (vocab, d), (h.dtype,), dev),
           _buf(target, "target", lead, (torch.int32,), dev))
    loss, pl = _out(loss, "loss", lead, torch.float32, h)
    lse, pz = _out(lse, "lse", lead, torch.float32, h)
    code = _DT[h.dtype]
    _run(_lib.poetx_xent_forward, dev, (n, d, vocab, code, *ins, pl, pz),
         (n, d, vocab, code, None, None, None, None, None))
    return loss, lse


def poetx_xent_backward(h: torch.Tensor, w: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                        dloss: torch.Tensor, *, want_dh: bool = True, want_dw: bool = True):
    """Gradients of sum(dloss * loss): dict with those of dh and dw that are wanted, in h's
    dtype.  lse: poetx_xent_forward's; dloss: float32, one per token (1 / count for a mean)."""
    n, d = _tokens(h, "h")
    dev = h.device
    vocab = w.shape[0]
    lead = h.shape[:-1]
    if not (want_dh or want_dw):
        raise ValueError("neither dh nor dw is wanted")
    ins = (_buf(h, "h", h.shape, _FLOATS, dev), _buf(w, "w", (vocab, d), (h.dtype,), dev),
           _buf(target, "target", lead, (torch.int32,), dev), _buf(lse, "lse", lead, _F32, dev),
           _buf(dloss, "dloss", lead, _F32, dev))
    out = {}
    if want_dh:
        out["dh"] = torch.empty_like(h)
    if want_dw:
        out["dw"] = torch.empty_like(w)
    if n == 0 and not want_dw:
        return out
    code = _DT[h.dtype]
    _run(_lib.poetx_xent_backward, dev,
         (n, d, vocab, code, *ins, out["dh"].data_ptr() if want_dh else None,
          out["dw"].data_ptr() if want_dw else None),
         (n, d, vocab, code, None, None, None, None, None, _SOME if want_dh else None, _SOME if want_dw else None))
    return out


# ---------------------------------------------------------------------------
# Operators of a fine-tuning step: gated feed-forward projections, clipped policy loss, gradient
# norm and clipping.
# ---------------------------------------------------------------------------
def poetx_glu_forward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, act="silu", *,
                      h: Optional[torch.Tensor] = None, save: bool = False):
    """act(x . w_gate^T) (x . w_up^T).  Returns (h, gate, up): gate and up, the two projections, for
    the backward when save is set, else None.  act: as in poetx_linear_forward."""
    n, d = _tokens(x, "x")
    dev, dt = x.device, (x.dtype,)
    f = w_gate.shape[0]
    a = _act(act)
    shape = x.shape[:-1] + (f,)
    ins = (_buf(x, "x", x.shape, _FLOATS, dev), _buf(w_gate, "w_gate", (f, d), dt, dev),
           _buf(w_up, "w_up", (f, d), dt, dev))
    h, ph = _out(h, "h", shape, x.dtype, x)
    gate = up = pg = pu = None
    if save:
        gate, up = torch.empty_like(h), torch.empty_like(h)
        pg, pu = gate.data_ptr(), up.data_ptr()
    code, some = _DT[x.dtype], _SOME if save else None
    _run(_lib.poetx_glu_forward, dev, (n, d, f, code, *ins, a, ph, pg, pu),
         (n, d, f, code, None, None, None, a, None, some, some))
    return h, gate, up


def poetx_glu_backward(x: Optional[torch.Tensor], w_gate: Optional[torch.Tensor], w_up: Optional[torch.Tensor],
                       dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, act="silu", *, want_dx: bool = True,
                       want_dw: bool = True):
    """Returns dict with those of dx and (dw_gate, dw_up) that are wanted, in dh's dtype.  gate, up:
    what poetx_glu_forward(save=True) returned.  x is needed for dw, the weights for dx."""
    n, f = _tokens(dh, "dh")
    dev, dt = dh.device, (dh.dtype,)
    a = _act(act)
    if not (want_dx or want_dw):
        raise ValueError("neither dx nor dw is wanted")
    if want_dx and (w_gate is None or w_up is None) or want_dw and x is None:
        raise ValueError("dx needs w_gate and w_up, dw needs x")
    if gate is None or up is None:
        raise ValueError("gate and up are required")
    d = (x if x is not None else w_gate).shape[-1]
    shape = dh.shape[:-1] + (d,)
    pdh = _buf(dh, "dh", dh.shape, _FLOATS, dev)
    ins = (_buf(x, "x", shape, dt, dev), _buf(w_gate, "w_gate", (f, d), dt, dev), _buf(w_up, "w_up", (f, d), dt, dev),
           pdh, _buf(gate, "gate", dh.shape, dt, dev), _buf(up, "up", dh.shape, dt, dev))
    out, ptrs = {}, [None, None, None]
    if want_dx:
        out["dx"] = dh.new_empty(shape)
        ptrs[0] = out["dx"].data_ptr()
    if want_dw:
        out["dw_gate"], out["dw_up"] = dh.new_empty((f, d)), dh.new_empty((f, d))
        ptrs[1:] = out["dw_gate"].data_ptr(), out["dw_up"].data_ptr()
    if n == 0 and not want_dw:
        return out
    code = _DT[dh.dtype]
    _run(_lib.poetx_glu_backward, dev, (n, d, f, code, *ins, a, *ptrs),
         (n, d, f, code, None, None, None, None, None, None, a, *(None if p is None else _SOME for p in ptrs)))
    return out


_REDUCE = {"token": POETX_REDUCE_TOKEN, "sequence": POETX_REDUCE_SEQUENCE, "sum": POETX_REDUCE_SUM}
_FLAGS = (torch.bool, torch.uint8)
_I64 = (torch.int64,)


@functools.lru_cache(maxsize=64)
def _policy(low: float, high: float, beta: float, scale: float, reduce: int, per_token: bool):
    """A pointer to the parameters, which it keeps alive."""
    return _byref(PoetxPolicyC(low, high, beta, scale, reduce, int(per_token)))


def poetx_policy_loss(nll: torch.Tensor, adv: torch.Tensor, offsets: Optional[torch.Tensor] = None, *,
                      nll_old: Optional[torch.Tensor] = None, nll_ref: Optional[torch.Tensor] = None,
                      mask: Optional[torch.Tensor] = None, per_token: bool = False, clip=(0.2, 0.2),
                      beta: float = 0.0, reduce: str = "token", scale: float = 1.0, want_grad: bool = True,
                      dnll: Optional[torch.Tensor] = None):
    """Clipped policy loss with a KL term on negative log-probabilities, float32, one per token
    (poetx_xent_forward's loss).  Returns (stats, dnll): stats float32 [4], loss, its policy part,
    the KL and the share of ratios held at a border; dnll the loss's gradient (None without
    want_grad), poetx_xent_backward's dloss.  adv: float32, one per sequence, or per token with
    per_token.  offsets: int64 [sequences + 1], where each sequence begins in nll's flat order and
    the last ends; None: one sequence of all tokens.  mask: bool or uint8 like nll, 0 for a token
    that does not count.  nll_old None: on-policy, ratio 1; nll_ref None: no KL.  reduce: "token",
    "sequence" or "sum"; clip: (low, high), the ratio's way below and above 1; scale: a factor of dnll."""
    dev, shape, n = nll.device, nll.shape, nll.numel()
    if reduce not in _REDUCE:
        raise ValueError(f"reduce: {reduce!r}, expected one of {tuple(_REDUCE)}")
    if beta != 0 and nll_ref is None:
        raise ValueError("beta needs nll_ref")
    low, high = clip
    seqs = 1
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected [sequences + 1]")
        seqs = offsets.numel() - 1
    ins = (_buf(offsets, "offsets", (seqs + 1,), _I64, dev), _buf(nll, "nll", shape, _F32, dev),
           _buf(nll_old, "nll_old", shape, _F32, dev), _buf(nll_ref, "nll_ref", shape, _F32, dev),
           _buf(adv, "adv", shape if per_token else (seqs,), _F32, dev), _buf(mask, "mask", shape, _FLAGS, dev))
    p = _policy(float(low), float(high), float(beta), float(scale), _REDUCE[reduce], bool(per_token))
    stats = nll.new_empty(4)
    pd = None
    if want_grad or dnll is not None:
        dnll, pd = _out(dnll, "dnll", None, torch.float32, nll)
    _run(_lib.poetx_policy_loss, dev, (n, seqs, *ins, p, stats.data_ptr(), pd),
         (n, seqs, None, None, None, None, None, _SOME if mask is not None else None, p, None, None))
    return stats, dnll


class GradList:
    """The gradients of a training step, for poetx_grad_norm and poetx_grad_clip: contiguous float32
    or bf16 tensors on one device, of any shapes.  out: where the clipped gradients go, tensors like
    them that share no memory with them; None: in place.  The list keeps its tensors (their memory
    must stay theirs: no resizing, no setting of .data); a program whose gradients stay where they are
    makes it once.  A list of more than 140 gradients keeps its device form (poetx_grad_plan) for each
    stream that it is used on."""

    def __init__(self, grads, out=None):
        self.grads = tuple(grads)
        self.out = None if out is None else tuple(out)
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError(f"out: {len(self.out)} tensors, expected {len(self.grads)}")
        if not self.grads:
            raise ValueError("no gradients")
        self.device = self.grads[0].device
        self.array = (PoetxGradC * len(self.grads))()
        for k, g in enumerate(self.grads):
            o = g if self.out is None else self.out[k]
            for t, name in ((g, f"gradient {k}"), (o, f"out {k}")):
                if t.dtype not in _FLOATS:
                    raise ValueError(f"{name}: dtype {t.dtype}, expected one of {_FLOATS}")
                if t.device != self.device:
                    raise ValueError(f"{name} is on {t.device}, expected {self.device}")
                if not t.is_contiguous():
                    raise ValueError(f"{name} must be contiguous")
            if o.dtype != g.dtype or o.shape != g.shape:
                raise ValueError(f"out {k}: {o.dtype} {tuple(o.shape)}, expected {g.dtype} {tuple(g.shape)}")
            self.array[k] = PoetxGradC(g.data_ptr(), o.data_ptr(), g.numel(), _DT[g.dtype])
        # every element is written once, and none that another gradient is read from
        spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                 for t in self.grads + (self.out or ()) if t.numel()]
        spans.sort()
        for (_, end), (begin, _) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError("gradients" + ("" if self.out is None else " and out") + " share memory")
        need, n = _sz(0), len(self.grads)
        _check(_lib.poetx_grad_plan(n, self.array, None, _byref(need), None), "poetx_grad_plan(size)")
        self._plan_bytes, self._plans = need.value, {}
        # with a plan where one is needed
        _check(_lib.poetx_grad_norm(n, self.array, 0.0, None, None, _SOME, None, _byref(need), None),
               "poetx_grad_norm(size)")
        self.workspace_bytes = need.value

    def plan(self) -> Optional[torch.Tensor]:
        """The list's device form for the current stream of its device, which is the current device
        (None: it needs none).  A call under graph capture makes its own, in the graph, from the
        graph's memory pool.  The caller holds the tensor until its kernels are launched, so that
        nothing it allocates before then takes the same memory."""
        if not self._plan_bytes:
            return None
        key, capturing = _raw_stream(self.device.index), _capturing()
        p = None if capturing else self._plans.get(key)
        if p is None:
            p = torch.empty(self._plan_bytes, dtype=torch.uint8, device=self.device)
            _check(_lib.poetx_grad_plan(len(self.grads), self.array, p.data_ptr(), _byref(_sz(self._plan_bytes)), key),
                   "poetx_grad_plan")
            if not capturing:
                self._plans[key] = p
        return p


def _grad_call(fn, grads, max_norm: float, out=None):
    if not isinstance(grads, GradList):
        grads = GradList(grads, out)
    elif out is not None:
        raise ValueError("out is the list's own")
    dev = grads.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on the GPU")
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return _grad_call(fn, grads, max_norm)
    r = torch.empty(2, dtype=torch.float32, device=dev)
    p, plan = r.data_ptr(), grads.plan()
    _run(fn, dev, (len(grads.grads), grads.array, max_norm, p, p + 4, None if plan is None else plan.data_ptr()),
         grads.workspace_bytes)
    del plan  # held until here
    return r[0], r[1]


def poetx_grad_norm(grads, max_norm: float = float("inf")):
    """(norm, coef), float32 scalars on the device: the norm of all gradients together, and the
    factor min(1, max_norm / norm) that clips them.  grads: a GradList or a sequence of tensors."""
    return _grad_call(_lib.poetx_grad_norm, grads, max_norm)


def poetx_grad_clip(grads, max_norm: float, out=None):
    """poetx_grad_norm, and the gradients times coef, in place or into out (a GradList has its
    own).  Returns (norm, coef)."""
    return _grad_call(_lib.poetx_grad_clip, grads, max_norm, out)


def prof_enable(on: bool = True):
    _check(_lib.poetx_prof_enable(1 if on else 0), "poetx_prof_enable")


def prof_only(label: Optional[str] = None):
    """Record only the launches labelled `label` (None: every launch)."""
    _check(_lib.poetx_prof_only(label.encode() if label else None), "poetx_prof_only")


def prof_read() -> dict:
    """{kernel label: (launches, total_ms, min_ms, max_ms)} recorded by this thread since
    the last read."""
    buf = ctypes.create_string_buffer(1 << 16)
    _check(_lib.poetx_prof_read(buf, len(buf)), "poetx_prof_read")
    out = {}
    for line in buf.value.decode().splitlines():
        name, n, ms, mn, mx = line.split()
        out[name] = (int(n), float(ms), float(mn), float(mx))
    return out


# Raw handle for tests of the host-side validation (calls that fail before any launch).
raw = _lib
