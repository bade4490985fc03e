"""Layer norm, forward and backward (``layer_norm_forward`` /
``layer_norm_backward`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
import functools
from array import array
from typing import Optional, Tuple

import torch
from torch import Tensor, empty_like

from . import _DTYPE, _lib, SeamBlendError
from ._call import call, like, written

_ptr = ctypes.c_void_p  # of shapes and strides too: places in one array.array
_lib.layer_norm_forward.argtypes = [_ptr, _ptr, _ptr, ctypes.c_float, _ptr, _ptr, ctypes.c_int, ctypes.c_int, _ptr,
                                    _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.layer_norm_forward.restype = ctypes.c_int
for _f in (_lib.layer_norm_forward_workspace_bytes, _lib.layer_norm_backward_workspace_bytes):
    _f.argtypes = [_ptr, ctypes.c_int]
    _f.restype = ctypes.c_size_t
_lib.layer_norm_backward.argtypes = [_ptr, _ptr, _ptr, _ptr, _ptr, ctypes.c_float, _ptr, ctypes.c_int,
                                     ctypes.c_int, _ptr, _ptr, _ptr, _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.layer_norm_backward.restype = ctypes.c_int
_DENSE = torch.contiguous_format
_F32 = torch.float32


def _rows(t: torch.Tensor, name: str):
    """(shape, dtype code) of a tensor of rows"""
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    shape = t.shape
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name} must have a last axis of at least one element")
    return shape, code


def _outer_axes(tensors):
    """The leading axes of tensors of one shape merged into at most two:
    (outer, inner, D), then each tensor's strides for the two."""
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
    pad = [0] * (2 - len(ext))
    return array("q", [1] * len(pad) + ext + [shape[-1]] + [v for s in strides for v in pad + s])


@functools.lru_cache(maxsize=256)
def _whole_rows(rows: int, d: int):
    a = array("q", (1, rows, d, 0, d, 0, d, 0, d))
    return a, a.buffer_info()[0]


def _geometry(rows: int, d: int, *tensors: torch.Tensor):
    """The library's shape and strides for tensors of one shape, in one array
    (with its address): the shape at its start, the k-th tensor's strides
    24 + 16 k bytes on."""
    for t in tensors:
        if not t.is_contiguous():
            a = _outer_axes(tensors)
            return a, a.buffer_info()[0]
    return _whole_rows(rows, d)


def _weight(t: torch.Tensor, name: str, d: int, x_dtype, index: int, dtype):
    """Checks one weight or its gradient; the dtype it shares with the others."""
    if not isinstance(t, Tensor) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on x's device")
    own = t.dtype
    if t.numel() != d or (own is not x_dtype and own is not _F32):
        raise ValueError(f"{name} must be [{d}] of x's dtype or float32")
    if dtype is not None and own is not dtype:
        raise ValueError("the weights and their gradients must be of one dtype")
    return own


def _like(t: torch.Tensor, name: str, shape, code: int, index: int):
    if _rows(t, name) != (shape, code) or t.get_device() != index:
        raise ValueError(f"{name} must match x")


_LONG = 16384  # rows of up to 64 KiB need no workspace


@functools.lru_cache(maxsize=256)
def _forward_workspace_bytes(rows: int, d: int, code: int) -> int:
    shape = array("q", (1, rows, d))
    n = _lib.layer_norm_forward_workspace_bytes(shape.buffer_info()[0], code)
    if n >> 63:
        raise SeamBlendError(-2, "layer_norm_forward_workspace_bytes")
    return max(16, n)


def _forward(x, gamma, beta, eps, out):
    """(out, device index, arguments of the library's call, what they point to)"""
    shape, code = _rows(x, "x")
    index, d, dtype, gp, bp = x.get_device(), shape[-1], None, None, None
    if gamma is not None:
        dtype, gp = _weight(gamma, "gamma", d, x.dtype, index, None), gamma.data_ptr()
    if beta is not None:
        dtype, bp = _weight(beta, "beta", d, x.dtype, index, dtype), beta.data_ptr()
    if out is None:
        out = empty_like(x, memory_format=_DENSE)
    else:
        _like(out, "out", shape, code, index)
    rows = x.numel() // d
    geometry, at = _geometry(rows, d, x, out)
    need, wp = 0, None
    if d > _LONG:  # such rows are split, their statistics merged through a workspace
        need = _forward_workspace_bytes(rows, d, code)
        geometry = (geometry, empty_like(like(index, need, torch.uint8), memory_format=_DENSE))
        wp = geometry[1].data_ptr()
    return out, index, (x.data_ptr(), at + 24, at, eps, gp, bp, code, code if dtype is None else _DTYPE[dtype],
                        out.data_ptr(), at + 40, wp, need), geometry


class LayerNorm:
    """A prepared layer norm call over fixed tensors (arguments validated and
    the output allocated once).  See layer_norm for the arguments."""

    def __init__(self, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, out: Optional[torch.Tensor] = None):
        self.out, _, self._args, geometry = _forward(x, gamma, beta, eps, out)
        self.device = x.device
        self._keep = (x, gamma, beta, geometry)

    def __call__(self) -> torch.Tensor:
        call(_lib.layer_norm_forward, "layer_norm_forward", self.device.index, self._args)
        written(self.out)
        return self.out


def layer_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
               eps: float = 1e-6, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Layer norm over the last axis of x (GPU tensor, fp32 / fp16 / bf16):
    ``(x - mean) / sqrt(var + eps) * gamma + beta``, statistics in fp32, rounded
    once.  The last axis must be contiguous; the others may be strided (views
    of a packed projection) as long as they merge into two.  gamma / beta: [D]
    of x's dtype or float32, or None.  ``out`` may be ``x``.  The result carries
    no autograd history: its gradient is layer_norm_backward."""
    y, index, args, geometry = _forward(x, gamma, beta, eps, out)
    call(_lib.layer_norm_forward, "layer_norm_forward", index, args)
    if out is not None:
        written(out)
    return y


@functools.lru_cache(maxsize=256)
def _workspace_bytes(index: int, rows: int, d: int, code: int) -> int:
    with torch.cuda.device(index):
        shape = array("q", (1, rows, d))
        n = _lib.layer_norm_backward_workspace_bytes(shape.buffer_info()[0], code)
    if n == 0:
        raise SeamBlendError(-1, "layer_norm_backward_workspace_bytes")
    return int(n)


def layer_norm_backward_workspace_bytes(x: torch.Tensor) -> int:
    """Bytes of workspace layer_norm_backward needs for x."""
    shape, code = _rows(x, "x")
    return _workspace_bytes(x.get_device(), x.numel() // shape[-1], shape[-1], code)


def _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace):
    """((dx, dgamma, dbeta), device index, arguments of the library's call, what they point to)"""
    shape, code = _rows(x, "x")
    index, d, x_dtype, dtype, gp = x.get_device(), shape[-1], x.dtype, None, None
    _like(dy, "dy", shape, code, index)
    if weight_grads is None:
        weight_grads = gamma is not None or dgamma is not None or dbeta is not None
    elif not weight_grads and (dgamma is not None or dbeta is not None):
        raise ValueError("dgamma or dbeta given with weight_grads=False")
    if gamma is not None:
        dtype, gp = _weight(gamma, "gamma", d, x_dtype, index, None), gamma.data_ptr()
    if dgamma is not None:
        dtype = _weight(dgamma, "dgamma", d, x_dtype, index, dtype)
    if dbeta is not None:
        dtype = _weight(dbeta, "dbeta", d, x_dtype, index, dtype)
    if weight_grads:
        if dtype is None:
            dtype = torch.float32
        if dgamma is None:
            dgamma = empty_like(like(index, d, dtype), memory_format=_DENSE)
        if dbeta is None:
            dbeta = empty_like(like(index, d, dtype), memory_format=_DENSE)
    if dx is None:
        dx = empty_like(x, memory_format=_DENSE)
    else:
        _like(dx, "dx", shape, code, index)
    rows = x.numel() // d
    if workspace is None:
        need = _workspace_bytes(index, rows, d, code)
        workspace = empty_like(like(index, need, torch.uint8), memory_format=_DENSE)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on x's device")
    else:
        need = workspace.numel() * workspace.element_size()
    geometry, at = _geometry(rows, d, dy, x, dx)
    return (dx, dgamma, dbeta), index, (
        dy.data_ptr(), at + 24, x.data_ptr(), at + 40, at, eps, gp, code, code if dtype is None else _DTYPE[dtype],
        dx.data_ptr(), at + 56, None if dgamma is None else dgamma.data_ptr(),
        None if dbeta is None else dbeta.data_ptr(), workspace.data_ptr(), need), (geometry, workspace)


class LayerNormBackward:
    """A prepared layer norm gradient over fixed tensors (arguments validated,
    outputs and workspace allocated once).  See layer_norm_backward."""

    def __init__(self, dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 dx: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                 dbeta: Optional[torch.Tensor] = None, weight_grads: Optional[bool] = None,
                 workspace: Optional[torch.Tensor] = None):
        self.out, _, self._args, keep = _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace)
        self.device = x.device
        self._keep = (dy, x, gamma, keep)

    def __call__(self) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
        call(_lib.layer_norm_backward, "layer_norm_backward", self.device.index, self._args)
        written(*self.out)
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
    GPU tensor of at least layer_norm_backward_workspace_bytes(x) bytes.  The
    results carry no autograd history."""
    out, index, args, keep = _backward(dy, x, gamma, eps, dx, dgamma, dbeta, weight_grads, workspace)
    call(_lib.layer_norm_backward, "layer_norm_backward", index, args)
    if dx is not None or dgamma is not None or dbeta is not None:
        written(dx, dgamma, dbeta)
    return out
