"""Dropout from a counter-based generator (``dropout_apply`` of
``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch
from torch import Tensor, empty_like

from . import _DTYPE, _lib
from ._call import call, written
from ._layer_norm import _geometry

_ptr = ctypes.c_void_p  # of shapes and strides too: places in one array.array
_lib.dropout_apply.argtypes = [_ptr, _ptr, _ptr, ctypes.c_int, ctypes.c_double, _ptr, ctypes.c_uint32, _ptr, _ptr, _ptr,
                               _ptr, _ptr]
_lib.dropout_apply.restype = ctypes.c_int
_DENSE = torch.contiguous_format


def _arguments(x, p, state, site, residual, out):
    """(out, device index, arguments of the library's call, what they point to)"""
    if isinstance(x, Tensor) and not x.dim():
        raise ValueError("x must have at least one axis")
    index = x.get_device() if isinstance(x, Tensor) and x.is_cuda else None
    if index is None:
        raise TypeError("x must be a GPU (HIP) tensor")
    code = _DTYPE.get(x.dtype)
    if code is None:
        raise TypeError(f"x: unsupported dtype {x.dtype}")
    if not isinstance(state, Tensor) or state.get_device() != index or state.dtype is not torch.int64 \
            or state.dim() != 1 or state.shape[0] != 2 or not state.is_contiguous():
        raise ValueError("state must be a contiguous int64 tensor of seed and offset on x's device")
    if not 0 <= site < 1 << 32:
        raise ValueError("site must be in 0..2^32")
    if out is None:
        out = empty_like(x, memory_format=_DENSE)
    for t, name in ((residual, "residual"), (out, "out")):
        if t is not None and (not isinstance(t, Tensor) or t.dtype is not x.dtype or t.get_device() != index
                              or t.shape != x.shape):
            raise ValueError(f"{name} must match x")
    # (without a residual its place repeats x's)
    three = (x, x if residual is None else residual, out)
    if x.is_contiguous() and out.is_contiguous() and (residual is None or residual.is_contiguous()):
        table, at = _geometry(1, x.numel(), *three)  # one row
    else:
        if x.shape[-1] < 1:
            raise ValueError("x must have a last axis of at least one element")
        table, at = _geometry(x.numel() // x.shape[-1], x.shape[-1], *three)
    return out, index, (x.data_ptr(), at + 24, at, code, p, state.data_ptr(), site,
                        None if residual is None else residual.data_ptr(), at + 40, out.data_ptr(), at + 56), table


class Dropout:
    """A prepared dropout over fixed tensors (arguments validated and the output
    allocated once).  See dropout for the arguments."""

    def __init__(self, x: torch.Tensor, p: float, state: torch.Tensor, site: int = 0,
                 residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
        self.out, _, self._args, table = _arguments(x, p, state, site, residual, out)
        self.device = x.device
        self._keep = (x, state, residual, table)

    def __call__(self) -> torch.Tensor:
        call(_lib.dropout_apply, "dropout_apply", self.device.index, self._args)
        written(self.out)
        return self.out


def dropout(x: torch.Tensor, p: float, state: torch.Tensor, site: int = 0, residual: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x / (1 - p) with a share p of its elements dropped, plus residual: GPU
    tensors of one shape and dtype (fp32 / fp16 / bf16), contiguous or strided
    before the last axis as long as those axes merge into two.  Which elements are
    dropped is a function of their index, of ``state`` (int64 GPU tensor: seed and
    offset, read when the kernel runs, so that a captured graph may move the
    offset) and of ``site`` (which of a step's dropouts this is); no mask is
    stored.  ``out`` may be ``x`` or ``residual``.  The result carries no autograd
    history: its gradient is dropout_backward with the same state and site."""
    y, index, args, table = _arguments(x, p, state, site, residual, out)
    call(_lib.dropout_apply, "dropout_apply", index, args)
    if out is not None:
        written(out)
    return y


def dropout_backward(dy: torch.Tensor, p: float, state: torch.Tensor, site: int = 0,
                     dx: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of dropout with respect to x (the residual's is dy itself): dy
    through the same mask, formed again from the state and site of the forward
    call.  ``dx`` may be ``dy``."""
    y, index, args, table = _arguments(dy, p, state, site, None, dx)
    call(_lib.dropout_apply, "dropout_apply", index, args)
    if dx is not None:
        written(dx)
    return y
