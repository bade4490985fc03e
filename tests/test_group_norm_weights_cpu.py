"""group_norm_backward refuses weight gradients that share memory with what it still
reads, or with each other, before any device work."""
from __future__ import annotations

import ctypes

import pytest

P = ctypes.c_void_p


def i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


@pytest.fixture(scope="module")
def lib():
    import seam_blending_patch_amd as sb
    return sb._lib


# [2, 6, 64] fp16, fp32 weights of 256 bytes each
@pytest.mark.parametrize("dgamma,dbeta,word", [
    (0x500000, 0xb00000, b"dgamma overlaps gamma"), (0x6000fc, 0xb00000, b"dgamma overlaps beta"),
    (0xa00000, 0x500000, b"dbeta overlaps gamma"), (0xa00000, 0x600000, b"dbeta overlaps beta"),
    (0xa00000, 0xa00000, b"dbeta overlaps dgamma"), (0xa00000, 0xa00004, b"dbeta overlaps dgamma"),
    (0xa00004, 0xa00000, b"dbeta overlaps dgamma"), (None, 0x5000fc, b"dbeta overlaps gamma"),
])
@pytest.mark.parametrize("positions", [6, 0])
def test_weight_gradients_that_overlap(lib, dgamma, dbeta, word, positions):
    rc = lib.group_norm_backward(P(0x900000), i64(384, 64), P(0x100000), i64(384, 64), i64(2, positions, 64), 4, P(0x700000),
                                 P(0x500000), P(0x600000), 1, 1, 0, P(0x200000), i64(384, 64), P(dgamma), P(dbeta),
                                 P(0x800000), 1 << 20, None)
    assert rc == -1 and word in lib.seamblend_last_error(), lib.seamblend_last_error()


def test_neighbours_are_no_overlap(lib):
    """weights next to each other in one buffer pass this check (and fail a later one, on
    purpose: a stride)"""
    rc = lib.group_norm_backward(P(0x900000), i64(384, 64), P(0x100000), i64(384, -64), i64(2, 6, 64), 4, P(0x700000),
                                 P(0x500000), P(0x500100), 1, 1, 0, P(0x200000), i64(384, 64), P(0x500200), P(0x500300),
                                 P(0x800000), 1 << 20, None)
    assert rc == -2 and b"strides of x" in lib.seamblend_last_error()
