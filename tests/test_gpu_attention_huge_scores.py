"""attention in fp16 with scores of 3.6e9, which fp32 holds in steps of 256: weights of one
binary order stay finite."""
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


@pytest.mark.parametrize("scale", [0.00566, 0.0058, 0.00588, 0.00604, 0.0061, 0.0075, 0.01])
@pytest.mark.parametrize("queries,d", [(1, 64), (40, 128), (300, 64), (140000, 128)])
def test_a_step_within_the_slack(sb, scale, queries, d):
    """64 keys of one score, 192 of 1024 more, which is less than what moves the running
    maximum; values tell them apart.  The two scores are exact, so their weights' ratio is
    off by the scale's rounding and an exponential's alone."""
    q, k, v = (torch.zeros(1, n, 1, d, dtype=torch.float16) for n in (queries, 256, 256))
    q[..., 0], q[..., 1], k[..., 0], k[:, 64:, :, 1], v[:, 64:] = 60000.0, 64.0, 60000.0, 16.0, 1.0
    out = sb.attention(q.cuda(), k.cuda(), v.cuda(), scale=scale)
    more = 192 * math.exp(1024 * scale)
    want = more / (64 + more)
    # The 192 keys' P are alike and rounded alike, by up to 2^-11 of themselves, while the sum
    # that divides them is not; the result is rounded by up to 2^-12 below 1; the weights'
    # ratio is off by its exponent's rounding, 2^-20 of a binary order
    assert (out.double() - want).abs().max().item() <= 2.0 ** -11 * want + 2.0 ** -12 + 2.0 ** -18
