"""Group norm of channels-last activations, forward and backward
(``group_norm_forward`` / ``group_norm_backward`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
import functools
from array import array
from typing import Optional, Tuple, Union

import torch
from torch import Tensor, empty_like

from . import _DTYPE, _lib, SeamBlendError
from ._call import call, like, written

_ptr = ctypes.c_void_p  # of shapes and strides too: places in one array.array
_int, _i64, _size = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_lib.group_norm_forward.argtypes = [_ptr, _ptr, _ptr, _i64, ctypes.c_float, _ptr, _ptr, _int, _int, _int, _ptr, _ptr,
                                    _ptr, _ptr, _size, _ptr]
_lib.group_norm_forward.restype = _int
_lib.group_norm_backward.argtypes = [_ptr, _ptr, _ptr, _ptr, _ptr, _i64, _ptr, _ptr, _ptr, _int, _int, _int, _ptr,
                                     _ptr, _ptr, _ptr, _ptr, _size, _ptr]
_lib.group_norm_backward.restype = _int
_lib.group_norm_workspace_bytes.argtypes = [_ptr, _i64, _int]
_lib.group_norm_workspace_bytes.restype = _size
_DENSE = torch.contiguous_format
_F32 = torch.float32
_ACTIVATIONS = {None: 0, "silu": 1}


def _positions(t: torch.Tensor, name: str):
    """(shape, dtype code) of a channels-last tensor"""
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() < 2 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be [N, ..., C] with at least one channel")
    return t.shape, code


def _strides(t: torch.Tensor, name: str):
    """(sample, position) strides: the axes between the first and the last merged"""
    shape, strides = t.shape, t.stride()
    if t.is_contiguous():
        c = shape[-1]
        return c * (t.numel() // (shape[0] * c) if t.numel() else 0), c
    if strides[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    step = None
    for n, s in zip(shape[-2:0:-1], strides[-2:0:-1]):  # innermost first
        if n == 1:
            continue
        if step is None:
            step, reach = s, s * n
        elif s != reach:
            raise ValueError(f"the axes of {name} between the first and the last must merge into one")
        else:
            reach *= n
    return strides[0] if shape[0] > 1 else 0, step or 0


def _weight(t: torch.Tensor, name: str, c: int, x_dtype, index: int, dtype):
    """Checks one weight or its gradient; the dtype it shares with the others."""
    if not isinstance(t, Tensor) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on x's device")
    own = t.dtype
    if t.numel() != c or (own is not x_dtype and own is not _F32):
        raise ValueError(f"{name} must be [{c}] of x's dtype or float32")
    if dtype is not None and own is not dtype:
        raise ValueError("the weights and their gradients must be of one dtype")
    return own


def _like(t: torch.Tensor, name: str, shape, code: int, index: int):
    if _positions(t, name) != (shape, code) or t.get_device() != index:
        raise ValueError(f"{name} must match x")


def _activation(activation) -> int:
    if activation not in _ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    return _ACTIVATIONS[activation]


def _stats(t: torch.Tensor, n: int, groups: int, index: int):
    if not isinstance(t, Tensor) or t.get_device() != index or t.dtype is not _F32 \
            or tuple(t.shape) != (n, groups, 3) or not t.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 tensor [{n}, {groups}, 3] on x's device")


@functools.lru_cache(maxsize=512)
def _workspace_bytes(index: int, n: int, s: int, c: int, groups: int, code: int) -> int:
    with torch.cuda.device(index):
        shape = array("q", (n, s, c))
        need = _lib.group_norm_workspace_bytes(shape.buffer_info()[0], groups, code)
    if need >> 63:
        raise SeamBlendError(-1, "group_norm_workspace_bytes")
    return need


def group_norm_workspace_bytes(x: torch.Tensor, groups: int) -> int:
    """Bytes of workspace group_norm and group_norm_backward need for x."""
    shape, code = _positions(x, "x")
    n, c = shape[0], shape[-1]
    return _workspace_bytes(x.get_device(), n, x.numel() // (n * c) if n else 0, c, groups, code)


def _workspace(workspace, index, n, s, c, groups, code):
    need = _workspace_bytes(index, n, s, c, groups, code)
    if workspace is None:
        workspace = empty_like(like(index, max(need, 16), torch.uint8), memory_format=_DENSE)
    elif not isinstance(workspace, Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on x's device")
    else:
        need = workspace.numel() * workspace.element_size()
    return workspace, need


def _forward(x, groups, gamma, beta, eps, activation, out, stats, return_stats, workspace):
    """((out, stats), device index, arguments of the library's call, what they point to)"""
    shape, code = _positions(x, "x")
    index, n, c, dtype, gp, bp = x.get_device(), shape[0], shape[-1], None, None, None
    act = _activation(activation)
    if gamma is not None:
        dtype, gp = _weight(gamma, "gamma", c, x.dtype, index, None), gamma.data_ptr()
    if beta is not None:
        dtype, bp = _weight(beta, "beta", c, x.dtype, index, dtype), beta.data_ptr()
    if out is None:
        out = empty_like(x, memory_format=_DENSE)
    else:
        _like(out, "out", shape, code, index)
    if stats is not None:
        _stats(stats, n, groups, index)
    elif return_stats:
        stats = torch.empty((n, groups, 3), dtype=_F32, device=x.device)
    s = x.numel() // (n * c) if n else 0
    workspace, need = _workspace(workspace, index, n, s, c, groups, code)
    table = array("q", (n, s, c, *_strides(x, "x"), *_strides(out, "out")))
    at = table.buffer_info()[0]
    return (out, stats), index, (
        x.data_ptr(), at + 24, at, groups, eps, gp, bp, act, code, code if dtype is None else _DTYPE[dtype],
        out.data_ptr(), at + 40, None if stats is None else stats.data_ptr(), workspace.data_ptr(), need), \
        (table, workspace)


class GroupNorm:
    """A prepared group norm over fixed tensors (arguments validated, output and
    workspace allocated once).  See group_norm for the arguments."""

    def __init__(self, x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
                 beta: Optional[torch.Tensor] = None, eps: float = 1e-6, activation: Optional[str] = None,
                 out: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None, return_stats: bool = False,
                 workspace: Optional[torch.Tensor] = None):
        (self.out, self.stats), _, self._args, keep = _forward(x, groups, gamma, beta, eps, activation, out, stats,
                                                               return_stats, workspace)
        self.device = x.device
        self._keep = (x, gamma, beta, keep)

    def __call__(self) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
        call(_lib.group_norm_forward, "group_norm_forward", self.device.index, self._args)
        written(self.out, self.stats)
        return self.out if self.stats is None else (self.out, self.stats)


def group_norm(x: torch.Tensor, groups: int, gamma: Optional[torch.Tensor] = None,
               beta: Optional[torch.Tensor] = None, eps: float = 1e-6, activation: Optional[str] = None,
               out: Optional[torch.Tensor] = None, stats: Optional[torch.Tensor] = None, return_stats: bool = False,
               workspace: Optional[torch.Tensor] = None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """Group norm of channels-last activations x [N, ..., C] (GPU tensor, fp32 /
    fp16 / bf16; a torch channels_last tensor is x.permute(0, 2, 3, 1)) with the
    activation behind it (None or "silu"): every group of C / groups channels of
    a sample is normed over all its positions, times gamma plus beta ([C] of x's
    dtype or float32, or None).  Statistics in fp32, rounded once.  The channels
    must be contiguous; the axes between may be strided as long as they merge into
    one.  ``out`` may be ``x``.  return_stats (or ``stats``, a float32 tensor
    [N, groups, 3] to write): returns (out, stats) with each group's mean as the sum
    of two numbers and 1 / sigma, which the gradient needs.  ``workspace``: optional
    uint8 GPU tensor of group_norm_workspace_bytes(x, groups) bytes.  The result
    carries no autograd history: its gradient is group_norm_backward."""
    (y, y_stats), index, args, keep = _forward(x, groups, gamma, beta, eps, activation, out, stats, return_stats,
                                               workspace)
    call(_lib.group_norm_forward, "group_norm_forward", index, args)
    if out is not None or stats is not None:
        written(out, stats)
    return y if y_stats is None else (y, y_stats)


def _backward(dy, x, groups, stats, gamma, beta, activation, dx, dgamma, dbeta, weight_grads, workspace):
    """((dx, dgamma, dbeta), device index, arguments of the library's call, what they point to)"""
    shape, code = _positions(x, "x")
    index, n, c, x_dtype, dtype, gp, bp = x.get_device(), shape[0], shape[-1], x.dtype, None, None, None
    act = _activation(activation)
    _like(dy, "dy", shape, code, index)
    _stats(stats, n, groups, index)
    if weight_grads is None:
        weight_grads = gamma is not None or beta is not None or dgamma is not None or dbeta is not None
    elif not weight_grads and (dgamma is not None or dbeta is not None):
        raise ValueError("dgamma or dbeta given with weight_grads=False")
    if gamma is not None:
        dtype, gp = _weight(gamma, "gamma", c, x_dtype, index, None), gamma.data_ptr()
    if beta is not None:
        dtype, bp = _weight(beta, "beta", c, x_dtype, index, dtype), beta.data_ptr()
    if dgamma is not None:
        dtype = _weight(dgamma, "dgamma", c, x_dtype, index, dtype)
    if dbeta is not None:
        dtype = _weight(dbeta, "dbeta", c, x_dtype, index, dtype)
    if weight_grads:
        if dtype is None:
            dtype = _F32
        if dgamma is None:
            dgamma = empty_like(like(index, c, dtype), memory_format=_DENSE)
        if dbeta is None:
            dbeta = empty_like(like(index, c, dtype), memory_format=_DENSE)
    if dx is None:
        dx = empty_like(x, memory_format=_DENSE)
    else:
        _like(dx, "dx", shape, code, index)
    s = x.numel() // (n * c) if n else 0
    workspace, need = _workspace(workspace, index, n, s, c, groups, code)
    table = array("q", (n, s, c, *_strides(dy, "dy"), *_strides(x, "x"), *_strides(dx, "dx")))
    at = table.buffer_info()[0]
    return (dx, dgamma, dbeta), index, (
        dy.data_ptr(), at + 24, x.data_ptr(), at + 40, at, groups, stats.data_ptr(), gp, bp, act, code,
        code if dtype is None else _DTYPE[dtype], dx.data_ptr(), at + 56,
        None if dgamma is None else dgamma.data_ptr(), None if dbeta is None else dbeta.data_ptr(),
        workspace.data_ptr(), need), (table, workspace)


class GroupNormBackward:
    """A prepared group norm gradient over fixed tensors (arguments validated,
    outputs and workspace allocated once).  See group_norm_backward."""

    def __init__(self, dy: torch.Tensor, x: torch.Tensor, groups: int, stats: torch.Tensor,
                 gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                 activation: Optional[str] = None, dx: Optional[torch.Tensor] = None,
                 dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                 weight_grads: Optional[bool] = None, workspace: Optional[torch.Tensor] = None):
        self.out, _, self._args, keep = _backward(dy, x, groups, stats, gamma, beta, activation, dx, dgamma, dbeta,
                                                  weight_grads, workspace)
        self.device = x.device
        self._keep = (dy, x, stats, gamma, beta, keep)

    def __call__(self) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
        call(_lib.group_norm_backward, "group_norm_backward", self.device.index, self._args)
        written(*self.out)
        return self.out


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, groups: int, stats: torch.Tensor,
                        gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                        activation: Optional[str] = None, dx: Optional[torch.Tensor] = None,
                        dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                        weight_grads: Optional[bool] = None, workspace: Optional[torch.Tensor] = None
                        ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradient of group_norm: (dx, dgamma, dbeta), from the forward call's input
    and its stats.  weight_grads: whether dgamma and dbeta (of the weights' dtype;
    float32 without any) are formed; by default where a weight or one of them is
    given, None in their place otherwise.  They are written, not added to,
    and share no memory with each other or a weight.
    ``dx`` may be ``dy`` or ``x``.  ``workspace``: optional uint8 GPU tensor of
    group_norm_workspace_bytes(x, groups) bytes.  The results carry no autograd
    history."""
    out, index, args, keep = _backward(dy, x, groups, stats, gamma, beta, activation, dx, dgamma, dbeta, weight_grads,
                                       workspace)
    call(_lib.group_norm_backward, "group_norm_backward", index, args)
    if dx is not None or dgamma is not None or dbeta is not None:
        written(dx, dgamma, dbeta)
    return out
