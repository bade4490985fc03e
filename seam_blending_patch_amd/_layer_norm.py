"""Layer norm, forward and backward (``layer_norm_forward`` /
``layer_norm_backward`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _DTYPE, _lib, SeamBlendError
from ._call import call

_i64 = ctypes.c_int64
_i64p = ctypes.POINTER(_i64)
_ptr = ctypes.c_void_p
_lib.layer_norm_forward.argtypes = [_ptr, _i64p, _i64p, ctypes.c_float, _ptr, _ptr, ctypes.c_int, ctypes.c_int, _ptr,
                                    _i64p, _ptr]
_lib.layer_norm_forward.restype = ctypes.c_int
_lib.layer_norm_backward_workspace_bytes.argtypes = [_i64p, ctypes.c_int]
_lib.layer_norm_backward_workspace_bytes.restype = ctypes.c_size_t
_lib.layer_norm_backward.argtypes = [_ptr, _i64p, _ptr, _i64p, _i64p, ctypes.c_float, _ptr, ctypes.c_int,
                                     ctypes.c_int, _ptr, _i64p, _ptr, _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.layer_norm_backward.restype = ctypes.c_int
_2 = _i64 * 2
_3 = _i64 * 3
_DENSE = torch.contiguous_format


def _require_rows(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must have a last axis of at least one element")


def _outer_axes(*tensors: torch.Tensor):
    """The leading axes of tensors of one shape merged into at most two:
    (outer, inner) extents and each tensor's strides for them."""
    shape = tensors[0].shape
    ext, strides = [], [[] for _ in tensors]
    for t in tensors:
        if t.stride(-1) != 1 and shape[-1] != 1:
            raise ValueError("the last axis must be contiguous")
    for k in range(len(shape) - 1):
        if shape[k] == 1:
            continue
        here = [t.stride(k) for t in tensors]
        if ext and all(s[-1] == h * shape[k] for s, h in zip(strides, here)):
            ext[-1] *= shape[k]
            for s, h in zip(strides, here):
                s[-1] = h
        else:
            ext.append(shape[k])
            for s, h in zip(strides, here):
                s.append(h)
    if len(ext) > 2:
        raise ValueError("the axes before the last must merge into at most two strided ones")
    pad = 2 - len(ext)
    return _3(*(1,) * pad, *ext, shape[-1]), [_2(*(0,) * pad, *s) for s in strides]


def _geometry(*tensors: torch.Tensor):
    """The library's shape and strides arguments for tensors of one shape."""
    for t in tensors:
        if not t.is_contiguous():
            return _outer_axes(*tensors)
    d = tensors[0].shape[-1]
    s = _2(0, d)
    return _3(1, tensors[0].numel() // d, d), (s,) * len(tensors)


def _weight(x: torch.Tensor, d: int, t: torch.Tensor, name: str, dtype):
    """Checks one weight or its gradient; the dtype it shares with the others."""
    if not isinstance(t, torch.Tensor) or t.get_device() != x.get_device() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on x's device")
    own = t.dtype
    if t.numel() != d or (own is not x.dtype and own is not torch.float32):
        raise ValueError(f"{name} must be [{d}] of x's dtype or float32")
    if dtype is not None and own is not dtype:
        raise ValueError("the weights and their gradients must be of one dtype")
    return own


def _like(x: torch.Tensor, t: torch.Tensor, name: str):
    _require_rows(t, name)
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must match x")


def _forward(x, gamma, beta, eps, out):
    """(out, arguments of the library's call)"""
    _require_rows(x, "x")
    d, dtype, gp, bp = x.shape[-1], None, None, None
    if gamma is not None:
        dtype, gp = _weight(x, d, gamma, "gamma", dtype), gamma.data_ptr()
    if beta is not None:
        dtype, bp = _weight(x, d, beta, "beta", dtype), beta.data_ptr()
    if out is None:
        out = torch.empty_like(x, memory_format=_DENSE)
    else:
        _like(x, out, "out")
    shape, (sx, so) = _geometry(x, out)
    code = _DTYPE[x.dtype]
    return out, (x.data_ptr(), sx, shape, eps, gp, bp, code, code if dtype is None else _DTYPE[dtype],
                 out.data_ptr(), so)


class LayerNorm:
    """A prepared layer norm call over fixed tensors (arguments validated and
    the output allocated once).  See layer_norm for the arguments."""

    def __init__(self, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, out: Optional[torch.Tensor] = None):
        self.out, self._args = _forward(x, gamma, beta, eps, out)
        self.device = x.device
        self._keep = (x, gamma, beta)

    def __call__(self) -> torch.Tensor:
        call(_lib.layer_norm_forward, "layer_norm_forward", self.device.index, self._args)
        return self.out


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Layer norm over the last axis of x (GPU tensor, fp32 / fp16 / bf16):
    ``(x - mean) / sqrt(var + eps) * gamma + beta``, statistics in fp32, rounded
    once.  The last axis must be contiguous; the others may be strided (views
    of a packed projection) as long as they merge into two.  gamma / beta: [D]
    of x's dtype or float32, or None.  ``out`` may be ``x``."""
    out, args = _forward(x, gamma, beta, eps, out)
    call(_lib.layer_norm_forward, "layer_norm_forward", x.get_device(), args)
    return out


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index: int, rows: int, d: int, code: int) -> int:
    with torch.cuda.device(index):
        n = _lib.layer_norm_backward_workspace_bytes(_3(1, rows, d), code)
    if n == 0:
        raise SeamBlendError(-1, "layer_norm_backward_workspace_bytes")
    return int(n)


def layer_norm_backward_workspace_bytes(x: torch.Tensor) -> int:
    """Bytes of workspace layer_norm_backward needs for x."""
    _require_rows(x, "x")
    d = x.shape[-1]
    return _workspace_bytes(x.get_device(), x.numel() // d, d, _DTYPE[x.dtype])


def _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace):
    """((dx, dgamma, dbeta), workspace, arguments of the library's call)"""
    _require_rows(x, "x")
    _like(x, dy, "dy")
    if weight_grads is None:
        weight_grads = gamma is not None or dgamma is not None or dbeta is not None
    elif not weight_grads and (dgamma is not None or dbeta is not None):
        raise ValueError("dgamma or dbeta given with weight_grads=False")
    d, dtype, gp = x.shape[-1], None, None
    if gamma is not None:
        dtype, gp = _weight(x, d, gamma, "gamma", dtype), gamma.data_ptr()
    if dgamma is not None:
        dtype = _weight(x, d, dgamma, "dgamma", dtype)
    if dbeta is not None:
        dtype = _weight(x, d, dbeta, "dbeta", dtype)
    if weight_grads:
        if dtype is None:
            dtype = torch.float32
        if dgamma is None:
            dgamma = x.new_empty(d, dtype=dtype)
        if dbeta is None:
            dbeta = x.new_empty(d, dtype=dtype)
    if dx is None:
        dx = torch.empty_like(x, memory_format=_DENSE)
    else:
        _like(x, dx, "dx")
    code = _DTYPE[x.dtype]
    need = _workspace_bytes(x.get_device(), x.numel() // d, d, code)
    if workspace is None:
        workspace = x.new_empty(need, dtype=torch.uint8)
    elif workspace.device != x.device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on x's device")
    else:
        need = workspace.numel() * workspace.element_size()
    shape, (sdy, sx, sdx) = _geometry(dy, x, dx)
    return (dx, dgamma, dbeta), workspace, (
        dy.data_ptr(), sdy, x.data_ptr(), sx, shape, eps, gp, code, code if dtype is None else _DTYPE[dtype],
        dx.data_ptr(), sdx, None if dgamma is None else dgamma.data_ptr(),
        None if dbeta is None else dbeta.data_ptr(), workspace.data_ptr(), need)


class LayerNormBackward:
    """A prepared layer norm gradient over fixed tensors (arguments validated,
    outputs and workspace allocated once).  See layer_norm_backward."""

    def __init__(self, dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                 dbeta: Optional[torch.Tensor] = None, weight_grads: Optional[bool] = None,
                 workspace: Optional[torch.Tensor] = None):
        self.out, workspace, self._args = _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace)
        self.device = x.device
        self._keep = (dy, x, gamma, workspace)

    def __call__(self) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
        call(_lib.layer_norm_backward, "layer_norm_backward", self.device.index, self._args)
        return self.out


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                        dbeta: Optional[torch.Tensor] = None, weight_grads: Optional[bool] = None,
                        workspace: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradient of layer_norm: (dx, dgamma, dbeta).  x is the forward call's
    input; nothing else is kept from it.  weight_grads: whether dgamma and dbeta
    (of gamma's dtype; float32 without gamma) are formed; by default where gamma
    or one of them is given, None in their place otherwise.  They are written,
    not added to.  ``dx`` may be ``dy`` or ``x``.  ``workspace``: optional uint8
    GPU tensor of at least layer_norm_backward_workspace_bytes(x) bytes."""
    out, workspace, args = _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace)
    call(_lib.layer_norm_backward, "layer_norm_backward", x.get_device(), args)
    return out
