"""How the transformer operators call the library: on the tensors' device, on
its current stream."""
from __future__ import annotations

import torch

from . import _check

_current_device = torch.cuda.current_device
# the current stream as a plain number, without a Stream object around it (2 us
# of a call of 7)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) \
    or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def call(function, name: str, index: int, args):
    """The library's function on device ``index`` and its current stream."""
    if index == _current_device():
        rc = function(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = function(*args, _raw_stream(index))
    if rc:
        _check(rc, name)
