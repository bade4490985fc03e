"""group_norm of a group that holds an infinity or a NaN: it has no deviation, and every
value of it, its statistics' last number and its gradient are NaN; others are as ever."""
from __future__ import annotations

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", [(1, 40, 32), (2, 9000, 32), (1, 70001, 20)], ids=str)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_its_group_is_nan(sb, dtype, shape, bad, at):
    gen = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2))
    groups, per = 4, shape[2] // 4
    clean = sb.group_norm(x, groups, return_stats=True)
    row = {"first": 0, "middle": shape[1] // 2, "last": -1}[at]
    x[0, row, 2 * per - 1 if at == "last" else per] = bad
    y, stats = sb.group_norm(x, groups, return_stats=True)
    hit = torch.zeros(shape[0], groups, dtype=torch.bool, device="cuda")
    hit[0, 1] = True
    dx = sb.group_norm_backward(dy, x, groups, stats)[0]
    for t in (y, dx):
        assert torch.equal(torch.isnan(t).view(shape[0], shape[1], groups, per).all(1).all(-1), hit)
        assert torch.equal(torch.isnan(t).view(shape[0], shape[1], groups, per).any(1).any(-1), hit)
    assert torch.equal(torch.isnan(stats[..., 2]), hit)
    assert torch.equal(stats[~hit], clean[1][~hit])
