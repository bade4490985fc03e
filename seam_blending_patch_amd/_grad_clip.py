"""The norm of a list of gradients and clipping by it (``grad_norm`` /
``grad_norm_clip`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional, Sequence

import torch
from torch.autograd.graph import increment_version

from . import _DTYPE, _lib, SeamBlendError
from ._call import call, like

_ptr = ctypes.c_void_p  # of the tables too, which are array.array's
_lib.grad_norm_workspace_bytes.argtypes = [_ptr, ctypes.c_int64]
_lib.grad_norm_workspace_bytes.restype = ctypes.c_size_t
_lib.grad_norm.argtypes = [_ptr, _ptr, _ptr, ctypes.c_int64, _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.grad_norm.restype = ctypes.c_int
_lib.grad_norm_clip.argtypes = [_ptr, _ptr, _ptr, _ptr, _ptr, ctypes.c_int64, ctypes.c_float, ctypes.c_float,
                                _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.grad_norm_clip.restype = ctypes.c_int


def _dense(t: torch.Tensor) -> bool:
    """Whether t's elements fill one run of memory, in whatever order."""
    run = 1
    for s, n in sorted((s, n) for s, n in zip(t.stride(), t.shape) if n != 1):
        if s != run:
            return False
        run *= n
    return True


def _table(tensors: Sequence[torch.Tensor], name: str, index: int):
    """Pointers and dtype codes of the tensors, checked, a pass over them for a
    property: a model has hundreds."""
    try:
        codes = array("i", [_DTYPE[t.dtype] for t in tensors])
        where = list(map(torch.Tensor.get_device, tensors))
        whole = list(map(torch.Tensor.is_contiguous, tensors))
        ptrs = array("Q", list(map(torch.Tensor.data_ptr, tensors)))
    except (AttributeError, KeyError, TypeError):
        codes = None
    if codes is None or where.count(index) != len(where):
        raise TypeError(f"{name} must be float32, float16 or bfloat16 tensors on one GPU")
    if False in whole and not all(w or _dense(t) for w, t in zip(whole, tensors)):
        raise ValueError(f"{name} must be dense")
    return ptrs, codes, whole


def _refuse_repeated(keep):
    """Raises where a tensor with elements is written to twice."""
    ptrs, _, numels, outs, *_ = keep
    written = [p for p, n in zip(ptrs if outs is None else outs, numels) if n]
    if len(set(written)) != len(written):
        raise ValueError("a tensor to be written is given twice")


def _at(a: array) -> int:
    return a.buffer_info()[0]


def _clip(grads, max_norm, eps, out):
    """(norm, outputs, device index, function, its name, its arguments, what they point to)"""
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients")
    if not isinstance(grads[0], torch.Tensor) or not grads[0].is_cuda:
        raise TypeError("grads must be GPU (HIP) tensors")
    index, n = grads[0].get_device(), len(grads)
    ptrs, codes, whole = _table(grads, "grads", index)
    numels = array("q", list(map(torch.Tensor.numel, grads)))
    outs = out_codes = None
    if out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError("one output for each gradient")
        outs, out_codes, out_whole = _table(out, "out", index)
        if [t.shape for t in grads] != [t.shape for t in out] or any(
                not (a and b) and g.stride() != o.stride() for a, b, g, o in zip(whole, out_whole, grads, out)):
            raise ValueError("each output must have its gradient's shape and strides")
        if out_codes != codes and any(a != b and b != 0 for a, b in zip(codes, out_codes)):
            raise ValueError("each output must be of its gradient's dtype or float32")
    need = _lib.grad_norm_workspace_bytes(_at(numels), n)
    if need == 0:
        raise SeamBlendError(-1, "grad_norm_workspace_bytes")
    work = torch.empty_like(like(index, need, torch.uint8), memory_format=torch.contiguous_format)
    norm = torch.empty_like(like(index, 1, torch.float32).squeeze(0))
    tail = (norm.data_ptr(), work.data_ptr(), need)
    keep = (ptrs, codes, numels, outs, out_codes, work)
    out = grads if out is None else out
    if max_norm is None:
        return norm, out, index, _lib.grad_norm, "grad_norm", (_at(ptrs), _at(numels), _at(codes), n, *tail), keep
    return norm, out, index, _lib.grad_norm_clip, "grad_norm_clip", (
        _at(ptrs), None if outs is None else _at(outs), _at(numels), _at(codes),
        None if outs is None else _at(out_codes), n, max_norm, eps, *tail), keep


class GradNormClip:
    """A prepared gradient norm (``max_norm`` None) or clip over fixed tensors:
    arguments validated, the norm and the workspace allocated once.  See
    grad_norm_clip for the arguments."""

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: Optional[float], eps: float = 1e-6,
                 out: Optional[Sequence[torch.Tensor]] = None):
        grads = list(grads)
        self.norm, self.out, index, self._function, self._name, self._args, keep = _clip(grads, max_norm, eps, out)
        self.device = torch.device("cuda", index)
        if max_norm is not None:
            _refuse_repeated(keep)
        self._keep = (grads, keep)
        self._written = [self.norm] if max_norm is None else [self.norm, *self.out]

    def __call__(self) -> torch.Tensor:
        call(self._function, self._name, self.device.index, self._args)
        increment_version(self._written)  # as torch counts its own writes
        return self.norm


def grad_norm(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """The 2-norm over every element of ``grads`` (dense GPU tensors, dtypes
    mixed as they come): a float32 scalar on the GPU, not waited for."""
    norm, _, index, function, name, args, keep = _clip(grads, None, 0.0, None)
    call(function, name, index, args)
    return norm


def grad_norm_clip(grads: Sequence[torch.Tensor], max_norm: float, eps: float = 1e-6,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales the gradients by ``min(1, max_norm / (norm + eps))``, norm the
    2-norm over all of them, in place or into ``out`` (tensors of the same shapes
    and strides, of the gradients' dtypes or float32: the 32-bit gradients an
    optimizer takes).  A tensor that is written may share memory with no other
    tensor of the call (refused).  Returns the norm before clipping, a float32 scalar on the
    GPU.  Nothing is waited for: a norm that is NaN or infinite shows in it and,
    as the formula says, in the gradients."""
    norm, out, index, function, name, args, keep = _clip(grads, max_norm, eps, out)
    try:
        call(function, name, index, args)
    except SeamBlendError:
        _refuse_repeated(keep)  # the library's answer to it is that they share memory
        raise
    increment_version(out)  # as torch counts its own writes
    return norm
