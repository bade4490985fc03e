"""CPU check of rotary_apply's limit on how far its positions reach: the kernel
forms their offsets in 64 bits."""
from __future__ import annotations

import ctypes

import pytest

P = ctypes.c_void_p
FAR = (1 << 40) - 1  # the longest stride taken


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.mark.parametrize("shape,strides,axes", [
    ((1, (1 << 12) + 2, 64), (0, 0, FAR), 1),
    ((1, (1 << 24) + 1, 64), (0, 0, FAR), 1),
    ((1 << 30, 1, 64), (0, FAR, 0), 1),
    ((1 << 12, 1 << 12, 64), (0, FAR, FAR), 2),
])
def test_positions_that_reach_too_far(shape, strides, axes):
    import seam_blending_patch_amd as sb
    lib = sb._lib
    st = i64(shape[1] * 64, 64, 64)
    rc = lib.rotary_apply(P(0x100000), st, P(1 << 45), st, 1, None, None, None, None, 0, i64(*shape), 0, P(0x3000000),
                          64, 0, P(0x3100000), 8, i64(*strides), i64(*([32] + [0] * (axes - 1))), axes, 1.0, 0, None)
    message = lib.seamblend_last_error()
    assert rc == -2 and message == b"positions span 2^52 elements or more", (rc, message)
