"""How the transformer operators call the library: on the tensors' device, on
its current stream."""
from __future__ import annotations

import functools

import torch
from torch.autograd.graph import increment_version

from . import _check

# the current device without a check that HIP is initialised: tensors are on it
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# the current stream as a plain number, without a Stream object around it (2 us
# of a call of 7)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) \
    or (lambda index: torch.cuda.current_stream(index).cuda_stream)


@functools.lru_cache(maxsize=512)
def like(index: int, n: int, dtype: torch.dtype) -> torch.Tensor:
    """n elements on a device that take the memory of one, to be given to
    torch.empty_like (half the time of torch.empty with a size and a dtype)."""
    return torch.empty(1, dtype=dtype, device=f"cuda:{index}").expand(n)


def call(function, name: str, index: int, args):
    """The library's function on device ``index`` and its current stream."""
    if index == _current_device():
        rc = function(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = function(*args, _raw_stream(index))
    if rc:
        _check(rc, name)


def written(*tensors):
    """Counts a caller's tensors (those that are not None) as written, as torch
    does for its own operations: a backward pass that saved one is refused
    instead of computed from what the call left in it."""
    increment_version([t for t in tensors if t is not None])
