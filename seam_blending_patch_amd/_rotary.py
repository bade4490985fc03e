"""Rotary position embedding (``rotary_apply`` of ``include/seam_blend.h``) and
the frequencies it turns by."""
from __future__ import annotations

import ctypes
import math
from array import array
from typing import Optional, Sequence, Tuple, Union

import torch
from torch import Tensor, empty_like

from . import _DTYPE, _lib
from ._call import call, written

_i64 = ctypes.c_int64
_ptr = ctypes.c_void_p  # of shapes, strides and sections too: places in one array.array
_lib.rotary_apply.argtypes = [_ptr, _ptr, _ptr, _ptr, _i64, _ptr, _ptr, _ptr, _ptr, _i64, _ptr, ctypes.c_int,
                              _ptr, _i64, ctypes.c_int, _ptr, ctypes.c_int, _ptr, _ptr, ctypes.c_int,
                              ctypes.c_float, ctypes.c_int, _ptr]
_lib.rotary_apply.restype = ctypes.c_int
_DENSE = torch.contiguous_format
_INTEGERS = (torch.int64, torch.int32)


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                       original_length: int = 0, low_turns: float = 1.0, high_turns: float = 32.0,
                       sections: Optional[Sequence[int]] = None, device="cuda") -> Tuple[torch.Tensor, float]:
    """Radians per position of the rot_dim / 2 pairs (float64 tensor on
    ``device``), and the factor for ``scale``.

    Pair i of n turns by ``base ** (-i / n)``; with ``sections`` (pair counts, one
    for each position axis) every section has a ladder of its own.  ``scaling``
    for contexts ``factor`` times longer:
      "linear"    f / factor (positions interpolated);
      "base"      base * factor ** (n / (n - 1)): the last pair is slowed by
                  factor, the first not at all;
      "by_parts"  pairs that turn more than high_turns times over
                  original_length are kept, those below low_turns slowed by
                  factor, those between mixed linearly in their turns; the
                  factor for ``scale`` is 0.1 ln(factor) + 1 (1 for a factor
                  up to 1).  Programs differ here: some mix linearly in the
                  pair's index, between two rounded ones, some scale by 1.  Give
                  weights tuned with such a program its own frequencies and scale.
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "by_parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    parts = (rot_dim // 2,) if sections is None else tuple(int(n) for n in sections)
    if any(n < 0 for n in parts) or sum(parts) != rot_dim // 2:
        raise ValueError("sections must add up to rot_dim / 2 pairs")
    if scaling == "base" and any(n == 1 for n in parts):
        raise ValueError("base scaling needs at least two pairs in a section")
    if scaling == "by_parts" and not (original_length > 0 and high_turns > low_turns):
        raise ValueError("by_parts scaling needs original_length > 0 and high_turns > low_turns")
    ladders = []
    for n in parts:
        b = base * factor ** (n / (n - 1)) if scaling == "base" and n else base
        ladders.append(b ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)))
    f = torch.cat(ladders)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "by_parts":
        turns = original_length * f / (2 * math.pi)
        keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return f.to(device), scale


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


def _output(like: torch.Tensor, shape, out: Optional[torch.Tensor], name: str):
    """(output, its strides)"""
    if out is None:
        out = empty_like(like, memory_format=_DENSE)
        s = out.stride()
        return out, s[:3] if len(s) == 4 else (0, s[0], s[1])
    out_shape, s = _heads(out, name)
    if out.dtype != like.dtype or out.device != like.device or out_shape != shape:
        raise ValueError(f"{name} must match {'k' if name == 'k_out' else 'q'}")
    return out, s


def _rotation(q, positions, freqs, k, interleaved, sections, scale, out, k_out, transpose):
    """(outputs, device index, arguments of the library's call, what they point to)"""
    shape, q_strides = _heads(q, "q")
    index, dtype = q.get_device(), q.dtype
    batch, length = (shape[0], shape[1]) if len(shape) == 4 else (1, shape[0])
    if not isinstance(freqs, Tensor) or freqs.get_device() != index or freqs.dtype is not torch.float64 \
            or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be a contiguous 1-D float64 tensor on q's device")
    if not isinstance(positions, Tensor) or positions.get_device() != index \
            or positions.dtype not in _INTEGERS:
        raise ValueError("positions must be an int64 or int32 tensor on q's device")
    pairs, ps, pn = freqs.numel(), positions.stride(), positions.shape
    if sections is None:
        parts, ps, pn = (pairs,), (0, *ps), (1, *pn)
    else:
        parts = tuple(sections)
    if len(pn) not in (2, 3) or pn[0] != len(parts) or pn[-1] != length or (len(pn) == 3 and pn[1] not in (1, batch)):
        raise ValueError("positions must be [T] or [B, T], with a leading axis for sections")
    out, out_strides = _output(q, shape, out, "out")
    # shape at 0, then strides of positions, q, its output, k, its output, then sections
    numbers = [batch, length, shape[-1], ps[0], ps[1] if len(ps) == 3 and pn[1] > 1 else 0, ps[-1], *q_strides,
               *out_strides]
    if k is None:
        if k_out is not None:
            raise ValueError("k_out without k")
        numbers += parts
        table = array("q", numbers)
        at = table.buffer_info()[0]
        k_args = (None, None, None, None, 0)
    else:
        k_shape, k_strides = _heads(k, "k")
        if k.dtype is not dtype or k.get_device() != index or k_shape[:-2] != shape[:-2] or k_shape[-1] != shape[-1]:
            raise ValueError("k must match q in all but its heads")
        k_out, k_out_strides = _output(k, k_shape, k_out, "k_out")
        numbers += k_strides
        numbers += k_out_strides
        numbers += parts
        table = array("q", numbers)
        at = table.buffer_info()[0]
        k_args = (k.data_ptr(), at + 96, k_out.data_ptr(), at + 120, k_shape[-2])
    n = len(parts)
    return (out if k is None else (out, k_out)), index, (
        q.data_ptr(), at + 48, out.data_ptr(), at + 72, shape[-2], *k_args, at, _DTYPE[dtype], freqs.data_ptr(),
        2 * pairs, 1 if interleaved else 0, positions.data_ptr(), positions.element_size(), at + 24,
        at + 8 * (len(numbers) - n), n, scale, 1 if transpose else 0), table


class Rotary:
    """A prepared rotation over fixed tensors (arguments validated and outputs
    allocated once).  See rotary for the arguments; ``transpose`` turns by the
    negative angles."""

    def __init__(self, q: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                 k: Optional[torch.Tensor] = None, interleaved: bool = False,
                 sections: Optional[Sequence[int]] = None, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, transpose: bool = False):
        self.out, _, self._args, table = _rotation(q, positions, freqs, k, interleaved, sections, scale, out, k_out,
                                                   transpose)
        self.device = q.device
        self._keep = (q, k, positions, freqs, table)

    def __call__(self) -> Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]:
        call(_lib.rotary_apply, "rotary_apply", self.device.index, self._args)
        written(*(self.out if isinstance(self.out, tuple) else (self.out,)))
        return self.out


def rotary(q: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, k: Optional[torch.Tensor] = None,
           interleaved: bool = False, sections: Optional[Sequence[int]] = None, scale: float = 1.0,
           out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Rotary position embedding of the heads of q, and of k in the same launch:
    [B, T, heads, D] or [T, heads, D] GPU tensors of one dtype, the last axis
    contiguous, the others strided as they come.  The first 2 * len(freqs)
    elements of every head turn in pairs (neighbours where ``interleaved``, else
    the two halves) by position * freqs (float64, see rotary_frequencies), times
    ``scale``; the rest is copied.  positions: int64 or int32 [T] or [B, T];
    with ``sections`` (pair counts) a leading axis holds the positions each
    section turns by.  ``out`` / ``k_out`` may be ``q`` / ``k``.  Returns the
    turned q, or (q, k), without autograd history: the gradient is
    rotary_backward."""
    turned, index, args, table = _rotation(q, positions, freqs, k, interleaved, sections, scale, out, k_out, False)
    call(_lib.rotary_apply, "rotary_apply", index, args)
    if out is not None or k_out is not None:
        written(out, k_out)
    return turned


def rotary_backward(dq: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor,
                    k: Optional[torch.Tensor] = None, interleaved: bool = False,
                    sections: Optional[Sequence[int]] = None, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
    """Gradient of rotary: the gradients of its outputs (dq, and k's as ``k``)
    turned back.  Arguments as rotary's."""
    turned, index, args, table = _rotation(dq, positions, freqs, k, interleaved, sections, scale, out, k_out, True)
    call(_lib.rotary_apply, "rotary_apply", index, args)
    if out is not None or k_out is not None:
        written(out, k_out)
    return turned
