"""Attention, forward and backward (``attention_forward`` /
``attention_backward`` of ``include/seam_blend.h``)."""
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
_int, _size, _float = ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_lib.attention_forward.argtypes = [_ptr] * 7 + [_int, _float, _int] + [_ptr] * 6 + [_size, _ptr]
_lib.attention_forward.restype = _int
_lib.attention_backward.argtypes = [_ptr] * 12 + [_int, _float, _int] + [_ptr] * 9 + [_size, _ptr]
_lib.attention_backward.restype = _int
for _f in (_lib.attention_forward_workspace_bytes, _lib.attention_backward_workspace_bytes):
    _f.argtypes = [_ptr, _int]
    _f.restype = _size
_DENSE = torch.contiguous_format
_F32, _I32 = torch.float32, torch.int32


def _heads(t: torch.Tensor, name: str):
    """(shape, strides [B, T, heads]) of a tensor of heads"""
    if not isinstance(t, Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a GPU (HIP) tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    shape, s = t.shape, t.stride()
    n = len(s)
    if n != 3 and n != 4:
        raise ValueError(f"{name} must be [B, T, heads, D] or [T, heads, D]")
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"the last axis of {name} must be contiguous")
    return shape, s[:3] if n == 4 else (0, s[0], s[1])


def _same(t: torch.Tensor, name: str, of: torch.Tensor, shape, as_name: str):
    """strides of a tensor of heads that has to be like another"""
    t_shape, strides = _heads(t, name)
    if t_shape != shape or t.dtype is not of.dtype or t.get_device() != of.get_device():
        raise ValueError(f"{name} must match {as_name}")
    return strides


def _output(t: Optional[torch.Tensor], name: str, of: torch.Tensor, shape, as_name: str):
    if t is None:
        t = empty_like(of, memory_format=_DENSE)
        s = t.stride()
        return t, s[:3] if len(s) == 4 else (0, s[0], s[1])
    return t, _same(t, name, of, shape, as_name)


def _lengths(t: Optional[torch.Tensor], name: str, batch: int, index: int):
    if t is None:
        return None
    if not isinstance(t, Tensor) or t.get_device() != index or t.dtype is not _I32 or t.dim() != 1 \
            or t.shape[0] != batch or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of one length a sample on q's device")
    return t.data_ptr()


def _statistics(t: torch.Tensor, shape, index: int):
    want = (shape[0], shape[2], shape[1]) if len(shape) == 4 else (shape[1], shape[0])
    if not isinstance(t, Tensor) or t.get_device() != index or t.dtype is not _F32 or tuple(t.shape) != want \
            or not t.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [B, heads, T] on q's device")


@functools.lru_cache(maxsize=512)
def _workspace_bytes(index: int, backward: bool, shape: tuple, code: int) -> int:
    of = _lib.attention_backward_workspace_bytes if backward else _lib.attention_forward_workspace_bytes
    with torch.cuda.device(index):
        table = array("q", shape)
        n = of(table.buffer_info()[0], code)
    if n >> 63:
        raise SeamBlendError(-2, "attention_backward_workspace_bytes" if backward
                             else "attention_forward_workspace_bytes")
    return n


def _sizes(q, k, v):
    """(index, dtype, (B, Lq, Lk, heads, key heads, D), q's, k's shapes, strides of q, k, v)"""
    shape, qs = _heads(q, "q")
    k_shape, ks = _heads(k, "k")
    if k.dtype is not q.dtype or k.get_device() != q.get_device() or len(k_shape) != len(shape) \
            or k_shape[-1] != shape[-1] or (len(shape) == 4 and k_shape[0] != shape[0]):
        raise ValueError("k must match q in all but its length and heads")
    vs = _same(v, "v", k, k_shape, "k")
    batch = shape[0] if len(shape) == 4 else 1
    return q.get_device(), q.dtype, (batch, shape[-3], k_shape[-3], shape[-2], k_shape[-2], shape[-1]), shape, \
        k_shape, (qs, ks, vs)


def _workspace(workspace, index, backward, sizes, code):
    """(what holds it, its address, its bytes)"""
    need = _workspace_bytes(index, backward, sizes, code)
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = empty_like(like(index, need, torch.uint8), memory_format=_DENSE)
    elif not isinstance(workspace, Tensor) or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on q's device")
    else:
        need = workspace.numel() * workspace.element_size()
    return workspace, workspace.data_ptr(), need


def _forward(q, k, v, causal, scale, query_lengths, key_lengths, out, lse, return_lse, workspace):
    """((out, lse), device index, arguments of the library's call, what they point to)"""
    index, dtype, sizes, shape, _, strides = _sizes(q, k, v)
    out, os = _output(out, "out", q, shape, "q")
    if lse is not None:
        _statistics(lse, shape, index)
    elif return_lse:
        lse = torch.empty((shape[0], shape[2], shape[1]) if len(shape) == 4 else (shape[1], shape[0]), dtype=_F32,
                          device=q.device)
    code = _DTYPE[dtype]
    held, wp, need = _workspace(workspace, index, False, sizes, code)
    table = array("q", (*sizes, *strides[0], *strides[1], *strides[2], *os))
    at = table.buffer_info()[0]
    return (out, lse), index, (
        q.data_ptr(), at + 48, k.data_ptr(), at + 72, v.data_ptr(), at + 96, at, code,
        sizes[5] ** -0.5 if scale is None else scale, 1 if causal else 0,
        _lengths(query_lengths, "query_lengths", sizes[0], index),
        _lengths(key_lengths, "key_lengths", sizes[0], index), out.data_ptr(), at + 120,
        None if lse is None else lse.data_ptr(), wp, need), (table, held)


class Attention:
    """A prepared attention call over fixed tensors (arguments validated, output
    and workspace allocated once): a decoding loop's, with key_lengths updated in
    place.  See attention for the arguments."""

    def __init__(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
                 scale: Optional[float] = None, query_lengths: Optional[torch.Tensor] = None,
                 key_lengths: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                 workspace: Optional[torch.Tensor] = None):
        (self.out, self.lse), _, self._args, keep = _forward(q, k, v, causal, scale, query_lengths, key_lengths, out,
                                                             lse, return_lse, workspace)
        self.device = q.device
        self._keep = (q, k, v, query_lengths, key_lengths, keep)

    def __call__(self) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
        call(_lib.attention_forward, "attention_forward", self.device.index, self._args)
        written(self.out, self.lse)
        return self.out if self.lse is None else (self.out, self.lse)


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False, scale: Optional[float] = None,
              query_lengths: Optional[torch.Tensor] = None, key_lengths: Optional[torch.Tensor] = None,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
              workspace: Optional[torch.Tensor] = None) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
    """softmax(scale q k^T) v: q [B, T, heads, D] or [T, heads, D], k and v
    [B, S, key heads, D] alike, GPU tensors of one dtype (fp32 / fp16 / bf16), the
    last axis contiguous, the others strided as they come; the query heads are a
    multiple of the key heads and share them in groups of neighbours; D up to 256.
    scale: D ** -0.5 by default.  ``causal``: query i sees keys up to
    i + (keys - queries).  query_lengths / key_lengths: int32 [B] GPU tensors of
    how many of each sample there are; what lies behind is not read, and its rows
    of the result are zeros.  A query that sees no key has zeros too.
    return_lse (or ``lse``, a float32 tensor [B, heads, T] to write): returns
    (out, lse) with the log of each row's sum of exponentials, which the
    gradient needs (-inf where no key is seen).  ``workspace``: optional uint8
    GPU tensor of attention_workspace_bytes(q, k) bytes.  The result carries no
    autograd history: its gradient is attention_backward."""
    (y, y_lse), index, args, keep = _forward(q, k, v, causal, scale, query_lengths, key_lengths, out, lse, return_lse,
                                             workspace)
    call(_lib.attention_forward, "attention_forward", index, args)
    if out is not None or lse is not None:
        written(out, lse)
    return y if y_lse is None else (y, y_lse)


def attention_workspace_bytes(q: torch.Tensor, k: torch.Tensor, backward: bool = False) -> int:
    """Bytes of workspace attention (attention_backward) needs for q and k."""
    index, dtype, sizes, _, _, _ = _sizes(q, k, k)
    return _workspace_bytes(index, backward, sizes, _DTYPE[dtype])


def _backward(dout, q, k, v, out, lse, causal, scale, query_lengths, key_lengths, dq, dk, dv, workspace):
    """((dq, dk, dv), device index, arguments of the library's call, what they point to)"""
    index, dtype, sizes, shape, k_shape, strides = _sizes(q, k, v)
    gs, os = _same(dout, "dout", q, shape, "q"), _same(out, "out", q, shape, "q")
    _statistics(lse, shape, index)
    dq, dqs = _output(dq, "dq", q, shape, "q")
    dk, dks = _output(dk, "dk", k, k_shape, "k")
    dv, dvs = _output(dv, "dv", v, k_shape, "v")
    code = _DTYPE[dtype]
    held, wp, need = _workspace(workspace, index, True, sizes, code)
    table = array("q", (*sizes, *gs, *strides[0], *strides[1], *strides[2], *os, *dqs, *dks, *dvs))
    at = table.buffer_info()[0]
    return (dq, dk, dv), index, (
        dout.data_ptr(), at + 48, q.data_ptr(), at + 72, k.data_ptr(), at + 96, v.data_ptr(), at + 120,
        out.data_ptr(), at + 144, lse.data_ptr(), at, code, sizes[5] ** -0.5 if scale is None else scale,
        1 if causal else 0, _lengths(query_lengths, "query_lengths", sizes[0], index),
        _lengths(key_lengths, "key_lengths", sizes[0], index), dq.data_ptr(), at + 168, dk.data_ptr(), at + 192,
        dv.data_ptr(), at + 216, wp, need), (table, held)


class AttentionBackward:
    """A prepared gradient of attention over fixed tensors (arguments validated,
    outputs and workspace allocated once).  See attention_backward."""

    def __init__(self, dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                 lse: torch.Tensor, causal: bool = False, scale: Optional[float] = None,
                 query_lengths: Optional[torch.Tensor] = None, key_lengths: Optional[torch.Tensor] = None,
                 dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                 dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
        self.out, _, self._args, keep = _backward(dout, q, k, v, out, lse, causal, scale, query_lengths, key_lengths,
                                                  dq, dk, dv, workspace)
        self.device = q.device
        self._keep = (dout, q, k, v, out, lse, query_lengths, key_lengths, keep)

    def __call__(self) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
        call(_lib.attention_backward, "attention_backward", self.device.index, self._args)
        written(*self.out)
        return self.out


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, causal: bool = False, scale: Optional[float] = None,
                       query_lengths: Optional[torch.Tensor] = None, key_lengths: Optional[torch.Tensor] = None,
                       dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradient of attention: (dq, dk, dv) from dout and the forward call's
    inputs and results (out, lse).  The probabilities are formed again, nothing of
    the scores' size is stored.  The gradients may be written into strided views
    (of a packed projection's gradient) given as dq, dk, dv; they are written, not
    added to, and share no memory with anything else.  Where lengths leave rows
    out those are zeros, and what dout holds there is not read.  ``workspace``:
    optional uint8 GPU tensor of attention_workspace_bytes(q, k, backward=True)
    bytes.  The results carry no autograd history."""
    grads, index, args, keep = _backward(dout, q, k, v, out, lse, causal, scale, query_lengths, key_lengths, dq, dk,
                                         dv, workspace)
    call(_lib.attention_backward, "attention_backward", index, args)
    if dq is not None or dk is not None or dv is not None:
        written(dq, dk, dv)
    return grads
