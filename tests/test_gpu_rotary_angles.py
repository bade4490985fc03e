"""Rotary angles next to a quarter, half and whole turn: a cosine or sine that is
small there is as exact, for its size, as any other."""
from __future__ import annotations

import math
import sys

import numpy as np
import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def cosines_and_sines(sb, freqs, positions):
    """Heads of first halves 1 and second halves 0 come out as (cos, sin)."""
    n = freqs.numel()
    q = torch.zeros(positions.numel(), 1, 2 * n, device="cuda")
    q[..., :n] = 1.0
    y = ref.f64(sb.rotary(q, positions, freqs))[:, 0]
    return y[:, :n], y[:, n:]


def allowed(want, angle):
    """cos a = cos r cos d - sin r sin d for the angle r that fp32 holds and the
    rest d: cos r is good to 2 ulp of itself (4 U) and exact where it is 0, d to
    4 U of itself, and the product and the sum round once each: 12 U of the sum of
    both terms' sizes.  fp32's neighbours of a quarter turn are at least 2 d from
    it, so that sum is at most 3 times the result: 36 U.  The 64-bit angle before
    that is off by less than 2^-50 of itself on either side."""
    return 36 * ref.U * np.abs(want) + 2.0 ** -50 * np.abs(angle)


@pytest.mark.parametrize("quarter", [-3, -2, -1, 0, 1, 2, 3, 4, 400001])
def test_small_cosines_and_sines(sb, quarter):
    off = np.array([s * v for v in (1e-3, 3e-5, 1e-6, 7e-8, 2e-8, 1e-8, 3e-9, 1e-10) for s in (1, -1)])
    freqs = torch.from_numpy(quarter * (math.pi / 2) + off).cuda()
    print(f"[rotary] {quarter} quarter turns", file=sys.stderr, flush=True)
    c, s = cosines_and_sines(sb, freqs, torch.ones(1, dtype=torch.int64, device="cuda"))
    angle = freqs.cpu().numpy()
    for got, want, name in ((c[0], np.cos(angle), "cosine"), (s[0], np.sin(angle), "sine")):
        assert (np.abs(got - want) <= allowed(want, angle)).all(), (name, got, want)


def test_error_over_a_turn_and_far_positions(sb):
    """Root mean square of the distance from (cos, sin): rounding both to fp32
    makes it 0.35 U, and the functions may add as much of their own, 0.5 U in
    all.  An angle rounded to fp32 would add 0.69 U: half of a turn's angles are
    then off by up to pi / 2 U, evenly spread."""
    freqs, _ = sb.rotary_frequencies(64)
    positions = torch.randint(1 << 20, (20000,), generator=torch.Generator().manual_seed(1)).cuda()
    c, s = cosines_and_sines(sb, freqs, positions)
    angle = ref.f64(positions)[:, None] * ref.f64(freqs)
    off = np.sqrt(((c - np.cos(angle)) ** 2 + (s - np.sin(angle)) ** 2).mean())
    print(f"[rotary] distance {off / ref.U:.3f} U", file=sys.stderr, flush=True)
    assert off <= 0.6 * ref.U
