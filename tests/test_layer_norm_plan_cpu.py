"""CPU check of which layer norm gradients one block takes: the workspace holds
a block of partials for each block."""
from __future__ import annotations

import ctypes

import pytest

F32, F16, BF16 = 0, 1, 2


def workspace(rows, d, dtype):
    import seam_blending_patch_amd as sb
    return sb._lib.layer_norm_backward_workspace_bytes((ctypes.c_int64 * 3)(1, rows, d), dtype)


@pytest.mark.parametrize("rows,d,dtype", [(16, 768, F32), (16, 2048, BF16), (8, 4096, BF16), (2, 8192, F16), (1, 16384, BF16)])
def test_short_rows_in_one_block(rows, d, dtype):
    assert workspace(rows, d, dtype) == workspace(1, d, dtype)


@pytest.mark.parametrize("rows,d,dtype", [(3, 8192, BF16), (4, 8192, F16), (2, 16384, BF16), (4, 16384, F16),
                                          (4, 10000, BF16), (3, 4096, F32), (4, 8192, F32)])
def test_long_rows_in_a_block_each(rows, d, dtype):
    """One block would take longer than the second launch costs."""
    assert workspace(rows, d, dtype) == rows * workspace(1, d, dtype)
