"""group_norm over groups that no block holds, where some value is far from the rest or
the mean is large: as exact as for any others."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import channels_ref as ref
from transformer_ref import U, assert_near, f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def check(sb, x, dy, groups, what):
    """No first value enters the bound: the statistics are off by CHAIN U of a deviation
    (a batch of 8 positions that holds a value D deviations out is off by some D U, and
    counts 8 / n in a group of n, where D is below the root of n), a value by as much of
    itself."""
    n, s, c = x.shape
    v = f64(x).reshape(n, s, groups, c // groups)
    mean = v.mean((1, 3), keepdims=True)
    r = 1 / np.sqrt(((v - mean) ** 2).mean((1, 3), keepdims=True) + EPS)
    h = ((v - mean) * r).reshape(x.shape)
    e_h = ref.CHAIN * U * (1 + np.abs(h))
    y, stats = sb.group_norm(x, groups, eps=EPS, return_stats=True)
    assert_near(y, h, e_h, what + " y")
    g = f64(dy)
    over = lambda t: np.broadcast_to(t.reshape(v.shape).mean((1, 3), keepdims=True), v.shape).reshape(x.shape)  # noqa: E731
    mg, mgh, r = over(g), over(g * h), np.broadcast_to(r, v.shape).reshape(x.shape)
    inner = g - mg - h * mgh
    tol = r * (ref.CHAIN * U * (over(np.abs(g)) + np.abs(h) * over(np.abs(g * h)) + np.abs(inner)) + over(np.abs(g) * e_h) * np.abs(h)
               + e_h * np.abs(mgh) + 4 * U * (np.abs(g) + np.abs(mg) + np.abs(h * mgh)))
    assert_near(sb.group_norm_backward(dy, x, groups, stats)[0], r * inner, tol, what + " dx")


SIZES = [((1, 9000, 24), 3), ((2, 12000, 8), 1), ((1, 70000, 32), 4), ((1, 9001, 13), 1), ((1, 30000, 20), 4)]


def draw(shape, dtype, mean=0.0):
    gen = torch.Generator().manual_seed(1)
    n = lambda: torch.randn(shape, generator=gen)  # noqa: E731
    return (n() + mean).to(DT[dtype]), n().to(DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape,groups", SIZES, ids=str)
@pytest.mark.parametrize("far", [200.0, 1e4, -6e4])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_a_value_far_out(sb, dtype, shape, groups, far, at):
    x, dy = draw(shape, dtype)
    x[:, {"first": 0, "middle": shape[1] // 2, "last": -1}[at], ::shape[2] // groups] = far
    check(sb, x.cuda(), dy.cuda(), groups, f"{shape} {dtype} {far} {at}")


@pytest.mark.parametrize("shape,groups", SIZES, ids=str)
@pytest.mark.parametrize("mean", [3000.0, -50.0])
def test_a_large_mean(sb, shape, groups, mean):
    x, dy = draw(shape, "fp32", mean)
    check(sb, x.cuda(), dy.cuda(), groups, f"{shape} {mean}")


@pytest.mark.parametrize("shape,groups", SIZES, ids=str)
def test_a_large_mean_and_a_first_value_of_zero(sb, shape, groups):
    x, dy = draw(shape, "fp32", 3000.0)
    x[:, 0] = 0.0
    check(sb, x.cuda(), dy.cuda(), groups, f"{shape}")


@pytest.mark.parametrize("shape,groups", SIZES, ids=str)
def test_the_mean_is_two_numbers(sb, shape, groups):
    x, _ = draw(shape, "fp32", 1000.0)
    _, stats = sb.group_norm(x.cuda(), groups, return_stats=True)
    v = f64(x).reshape(shape[0], shape[1], groups, -1)
    mean, s = v.mean((1, 3)), f64(stats)
    assert np.abs(s[..., 0] - mean).max() <= 1001 * U  # the mean in fp32 itself
    assert np.abs(s[..., 0] + s[..., 1] - mean).max() <= ref.CHAIN * U * v.std()


def test_constant_groups(sb):
    x = torch.full((1, 9000, 16), 7.3, device="cuda")
    y, stats = sb.group_norm(x, 2, return_stats=True)
    assert not y.any() and torch.equal(stats[..., 0], x[:, 0, :2]) and not stats[..., 1].any()
