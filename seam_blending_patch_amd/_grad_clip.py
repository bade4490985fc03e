"""The norm of a list of gradients and clipping by it (``grad_norm`` /
``grad_norm_clip`` of ``include/seam_blend.h``)."""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _DTYPE, _check, _lib, _stream_ptr, SeamBlendError

_i64p = ctypes.POINTER(ctypes.c_int64)
_intp = ctypes.POINTER(ctypes.c_int)
_ptr = ctypes.c_void_p
_ptrp = ctypes.POINTER(ctypes.c_void_p)
_lib.grad_norm_workspace_bytes.argtypes = [_i64p, ctypes.c_int64]
_lib.grad_norm_workspace_bytes.restype = ctypes.c_size_t
_lib.grad_norm.argtypes = [_ptrp, _i64p, _intp, ctypes.c_int64, _ptr, _ptr, ctypes.c_size_t, _ptr]
_lib.grad_norm.restype = ctypes.c_int
_lib.grad_norm_clip.argtypes = [_ptrp, _ptrp, _i64p, _intp, _intp, ctypes.c_int64, ctypes.c_float, ctypes.c_float,
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


def _table(tensors: Sequence[torch.Tensor], name: str, device):
    codes = []
    for t in tensors:
        if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPE or t.device != device:
            raise TypeError(f"{name} must be float32, float16 or bfloat16 tensors on one GPU")
        if not t.is_contiguous() and not _dense(t):
            raise ValueError(f"{name} must be dense")
        codes.append(_DTYPE[t.dtype])
    n = len(codes)
    return (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors]), (ctypes.c_int * n)(*codes)


class GradNormClip:
    """A prepared gradient norm (``max_norm`` None) or clip over fixed tensors:
    arguments validated, the norm and the workspace allocated once.  See
    grad_norm_clip for the arguments."""

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: Optional[float], eps: float = 1e-6,
                 out: Optional[Sequence[torch.Tensor]] = None):
        grads = list(grads)
        if not grads:
            raise ValueError("no gradients")
        dev = grads[0].device
        if dev.type != "cuda":
            raise TypeError("grads must be GPU (HIP) tensors")
        ptrs, codes = _table(grads, "grads", dev)
        n = len(grads)
        numels = (ctypes.c_int64 * n)(*[t.numel() for t in grads])
        outs = out_codes = None
        if out is not None:
            out = list(out)
            if len(out) != n:
                raise ValueError("one output for each gradient")
            outs, out_codes = _table(out, "out", dev)
            for g, o in zip(grads, out):
                if g.shape != o.shape or (g.stride() != o.stride() and not (g.is_contiguous() and o.is_contiguous())):
                    raise ValueError("each output must have its gradient's shape and strides")
                if o.dtype is not g.dtype and o.dtype is not torch.float32:
                    raise ValueError("each output must be of its gradient's dtype or float32")
        need = _lib.grad_norm_workspace_bytes(numels, n)
        if need == 0:
            raise SeamBlendError(-1, "grad_norm_workspace_bytes")
        work = torch.empty(need // 4 + 4, dtype=torch.float32, device=dev)
        self.norm, self.device, self.out = work[need // 4], dev, (grads if out is None else out)
        self._keep = (grads, work)
        tail = (self.norm.data_ptr(), work.data_ptr(), need)
        if max_norm is None:
            self._call, self._name, self._args = _lib.grad_norm, "grad_norm", (ptrs, numels, codes, n, *tail)
        else:
            self._call, self._name = _lib.grad_norm_clip, "grad_norm_clip"
            self._args = (ptrs, outs, numels, codes, out_codes, n, max_norm, eps, *tail)

    def __call__(self) -> torch.Tensor:
        _check(self._call(*self._args, _stream_ptr(self.device)), self._name)
        return self.norm


def grad_norm(grads: Sequence[torch.Tensor]) -> torch.Tensor:
    """The 2-norm over every element of ``grads`` (dense GPU tensors, dtypes
    mixed as they come): a float32 scalar on the GPU, not waited for."""
    plan = GradNormClip(grads, None)
    with torch.cuda.device(plan.device):
        return plan()


def grad_norm_clip(grads: Sequence[torch.Tensor], max_norm: float, eps: float = 1e-6,
                   out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Scales the gradients by ``min(1, max_norm / (norm + eps))``, norm the
    2-norm over all of them, in place or into ``out`` (tensors of the same shapes
    and strides, of the gradients' dtypes or float32: the 32-bit gradients an
    optimizer takes).  Returns the norm before clipping, a float32 scalar on the
    GPU.  Nothing is waited for: a norm that is NaN or infinite shows in it and,
    as the formula says, in the gradients."""
    plan = GradNormClip(grads, max_norm, eps, out)
    with torch.cuda.device(plan.device):
        return plan()
