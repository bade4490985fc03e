"""Layer norm, forward and backward (``layer_norm_forward`` /
``layer_norm_backward`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _DTYPE, _check, _lib, _stream_ptr, SeamBlendError

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
    if all(t.is_contiguous() for t in tensors):
        d = shape[-1]
        return (1, tensors[0].numel() // d), [(0, d)] * len(tensors)
    for t in tensors:
        if t.stride(-1) != 1 and shape[-1] != 1:
            raise ValueError("the last axis must be contiguous")
    ext, strides = [], [[] for _ in tensors]
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
    return (1,) * pad + tuple(ext), [(0,) * pad + tuple(s) for s in strides]


def _weights(x: torch.Tensor, **weights):
    """The dtype code of the weights given (x's where there are none)."""
    dtype = None
    for name, t in weights.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.device != x.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor on x's device")
        if t.numel() != x.shape[-1] or t.dtype not in (x.dtype, torch.float32):
            raise ValueError(f"{name} must be [{x.shape[-1]}] of x's dtype or float32")
        if dtype is not None and t.dtype != dtype:
            raise ValueError("the weights and their gradients must be of one dtype")
        dtype = t.dtype
    return _DTYPE[x.dtype if dtype is None else dtype]


def _like(x: torch.Tensor, t: torch.Tensor, name: str):
    _require_rows(t, name)
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must match x")


def _data(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


class LayerNorm:
    """A prepared layer norm call over fixed tensors (arguments validated and
    the output allocated once).  See layer_norm for the arguments."""

    def __init__(self, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, out: Optional[torch.Tensor] = None):
        _require_rows(x, "x")
        wdtype = _weights(x, gamma=gamma, beta=beta)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _like(x, out, "out")
        ext, (sx, so) = _outer_axes(x, out)
        self.out, self.device = out, x.device
        self._keep = (x, gamma, beta)
        self._args = (x.data_ptr(), _2(*sx), _3(*ext, x.shape[-1]), eps, _data(gamma), _data(beta), _DTYPE[x.dtype],
                      wdtype, out.data_ptr(), _2(*so))

    def __call__(self) -> torch.Tensor:
        _check(_lib.layer_norm_forward(*self._args, _stream_ptr(self.device)), "layer_norm_forward")
        return self.out


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Layer norm over the last axis of x (GPU tensor, fp32 / fp16 / bf16):
    ``(x - mean) / sqrt(var + eps) * gamma + beta``, statistics in fp32, rounded
    once.  The last axis must be contiguous; the others may be strided (views
    of a packed projection) as long as they merge into two.  gamma / beta: [D]
    of x's dtype or float32, or None.  ``out`` may be ``x``."""
    plan = LayerNorm(x, gamma, beta, eps, out)
    with torch.cuda.device(plan.device):
        return plan()


def layer_norm_backward_workspace_bytes(x: torch.Tensor) -> int:
    """Bytes of workspace layer_norm_backward needs for x."""
    _require_rows(x, "x")
    d = x.shape[-1]
    with torch.cuda.device(x.device):
        n = _lib.layer_norm_backward_workspace_bytes(_3(1, x.numel() // d, d), _DTYPE[x.dtype])
    if n == 0:
        raise SeamBlendError(-1, "layer_norm_backward_workspace_bytes")
    return int(n)


class LayerNormBackward:
    """A prepared layer norm gradient over fixed tensors (arguments validated,
    outputs and workspace allocated once).  See layer_norm_backward."""

    def __init__(self, dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                 dbeta: Optional[torch.Tensor] = None, weight_grads: Optional[bool] = None,
                 workspace: Optional[torch.Tensor] = None):
        _require_rows(x, "x")
        _like(x, dy, "dy")
        if weight_grads is None:
            weight_grads = gamma is not None or dgamma is not None or dbeta is not None
        wdtype = _weights(x, gamma=gamma, dgamma=dgamma, dbeta=dbeta)
        if weight_grads:
            given = next((t for t in (gamma, dgamma, dbeta) if t is not None), None)
            wt = torch.float32 if given is None else given.dtype
            wdtype = _DTYPE[wt]
            if dgamma is None:
                dgamma = torch.empty(x.shape[-1], dtype=wt, device=x.device)
            if dbeta is None:
                dbeta = torch.empty(x.shape[-1], dtype=wt, device=x.device)
        elif dgamma is not None or dbeta is not None:
            raise ValueError("dgamma or dbeta given with weight_grads=False")
        if dx is None:
            dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        else:
            _like(x, dx, "dx")
        need = layer_norm_backward_workspace_bytes(x)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        elif workspace.device != x.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous GPU tensor on x's device")
        ext, (sdy, sx, sdx) = _outer_axes(dy, x, dx)
        self.out, self.device = (dx, dgamma, dbeta), x.device
        self._keep = (dy, x, gamma, workspace)
        self._args = (dy.data_ptr(), _2(*sdy), x.data_ptr(), _2(*sx), _3(*ext, x.shape[-1]), eps, _data(gamma),
                      _DTYPE[x.dtype], wdtype, dx.data_ptr(), _2(*sdx), _data(dgamma), _data(dbeta),
                      workspace.data_ptr(), workspace.numel() * workspace.element_size())

    def __call__(self) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
        _check(_lib.layer_norm_backward(*self._args, _stream_ptr(self.device)), "layer_norm_backward")
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
    plan = LayerNormBackward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace)
    with torch.cuda.device(plan.device):
        return plan()
