"""group_norm and group_norm_backward against their definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import channels_ref as ref
from transformer_ref import assert_near, f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def draw(seed, shape, dtype, weights="fp32", mean=0.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    c = shape[-1]
    x = (n(*shape) * (0.3 + n(c).abs()) + n(c) + mean).to(DT[dtype]).cuda()
    dy = n(*shape).to(DT[dtype]).cuda()
    if weights == "none":
        return x, dy, None, None
    wt = torch.float32 if weights == "fp32" else DT[dtype]
    return x, dy, (1 + 0.3 * n(c)).to(wt).cuda(), (0.3 * n(c)).to(wt).cuda()


def flat(t):
    return None if t is None else f64(t).reshape(t.shape[0], -1, t.shape[-1]) if t.dim() > 1 else f64(t)


def check(sb, x, dy, gamma, beta, groups, act, what):
    silu = act == "silu"
    want, tol = ref.group_norm(flat(x), groups, flat(gamma), flat(beta), EPS, silu)
    y, stats = sb.group_norm(x, groups, gamma, beta, eps=EPS, activation=act, return_stats=True)
    assert_near(y, want.reshape(x.shape), tol.reshape(x.shape), what + " y")
    want, tol = ref.group_norm_backward(flat(dy), flat(x), groups, flat(gamma), flat(beta), EPS, silu)
    got = sb.group_norm_backward(dy, x, groups, stats, gamma, beta, activation=act, weight_grads=True)
    assert_near(got[0], want[0].reshape(x.shape), tol[0].reshape(x.shape), what + " dx")
    assert_near(got[1], want[1], tol[1], what + " dgamma")
    assert_near(got[2], want[2], tol[2], what + " dbeta")
    return y, stats, got


SIZES = [
    # [N, positions, C], groups
    ((1, 1, 1), 1), ((2, 1, 8), 4), ((1, 2, 64), 32), ((3, 33, 96), 32), ((1, 257, 320), 32), ((2, 64, 7), 7),
    ((1, 100, 13), 1), ((1, 1000, 4), 2), ((2, 50, 1280), 32), ((1, 9, 2049), 3), ((1, 20, 4100), 4), ((5, 17, 30), 10),
    ((1, 3001, 24), 8), ((2, 40, 2048), 16), ((130, 3, 16), 2),
    # at and past what a block holds of a group, forward (8192 vectors) and backward (5120)
    ((2, 1024, 320), 32), ((1, 4096, 64), 4), ((1, 4097, 64), 4), ((3, 1280, 128), 4), ((1, 1281, 128), 4), ((2, 1551, 96), 32),
    ((1, 8192, 16), 2), ((1, 8193, 16), 2), ((1, 900, 40), 4), ((1, 5120, 24), 3), ((2, 12000, 8), 1), ((1, 3, 4096), 1),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape,groups", SIZES, ids=str)
@pytest.mark.parametrize("act", [None, "silu"])
def test_sizes(sb, dtype, shape, groups, act):
    check(sb, *draw(1, shape, dtype), groups, act, f"{shape} {groups} {dtype}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("weights", ["none", "same", "fp32"])
def test_weights(sb, dtype, weights):
    check(sb, *draw(2, (2, 5, 7, 64), dtype, weights), 16, "silu", weights)
    x, dy, gamma, beta = draw(2, (2, 5, 7, 64), dtype, weights)
    if gamma is not None:
        check(sb, x, dy, gamma, None, 16, "silu", "gamma alone")
        check(sb, x, dy, None, beta, 16, "silu", "beta alone")
    _, stats = sb.group_norm(x, 16, return_stats=True)
    assert sb.group_norm_backward(dy, x, 16, stats)[1:] == (None, None)
    with pytest.raises(ValueError):
        sb.group_norm_backward(dy, x, 16, stats, weight_grads=False, dgamma=torch.empty(64, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("mean", [3000.0, -50.0])
def test_a_mean_that_is_large_against_the_spread(sb, dtype, mean):
    check(sb, *draw(3, (2, 300, 64), dtype, mean=mean), 8, "silu", str(mean))


def test_a_first_value_far_out(sb):
    """the sums' shift is no typical value of its group"""
    x, dy, gamma, beta = draw(4, (1, 400, 32), "fp32")
    x[0, 0, ::4] = 200.0
    check(sb, x, dy, gamma, beta, 8, None, "far")


def test_constant_groups(sb):
    x = torch.full((2, 30, 16), 7.0, device="cuda")
    gamma, beta = torch.full((16,), 2.0, device="cuda"), torch.linspace(-1, 1, 16, device="cuda")
    y, stats = sb.group_norm(x, 4, gamma, beta, return_stats=True)
    assert torch.equal(y, beta.expand_as(y))
    assert torch.equal(stats[..., 0] + stats[..., 1], torch.full((2, 4), 7.0, device="cuda"))
    dx, _, dbeta = sb.group_norm_backward(torch.ones_like(x), x, 4, stats, gamma, beta)
    assert torch.isfinite(dx).all() and torch.equal(dbeta, torch.full((16,), 60.0, device="cuda"))


def test_large_activations_do_not_overflow(sb):
    x, dy, _, beta = draw(5, (1, 40, 32), "fp32")
    check(sb, x, dy, torch.full((32,), 60.0, device="cuda"), beta, 4, "silu", "steep")
    x[0, 3, 0] = float("nan")
    y = sb.group_norm(x, 4)
    assert torch.isnan(y[..., :8]).all() and torch.isfinite(y[..., 8:]).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("c", [32, 30, 5])
def test_views_and_in_place(sb, dtype, c):
    """channels of wider positions, samples apart, odd offsets, torch's channels_last"""
    whole = draw(6, (3, 6, 9, c + 7), dtype, "none")[0]
    x = whole[::2, :, :, 3:c + 3]
    _, dy, gamma, beta = draw(7, x.shape, dtype)
    y, stats, grads = check(sb, x, dy, gamma, beta, 5 if c % 2 else 2, "silu", "view")
    groups = 5 if c % 2 else 2
    nchw = x.contiguous().permute(0, 3, 1, 2)
    assert torch.equal(sb.group_norm(nchw.permute(0, 2, 3, 1), groups, gamma, beta, activation="silu"), y)
    before = whole.clone()
    out = sb.group_norm(x, groups, gamma, beta, activation="silu", out=x)
    assert out is x and torch.equal(x, y)
    rest = torch.ones_like(whole, dtype=torch.bool)
    rest[::2, :, :, 3:c + 3] = False
    assert torch.equal(whole[rest], before[rest])
    x = before[::2, :, :, 3:c + 3]
    for into in (dy.clone(), x.contiguous()):
        got = sb.group_norm_backward(into if into.equal(dy) else dy, x if into.equal(dy) else into, groups, stats, gamma,
                                     beta, activation="silu", dx=into)
        assert got[0] is into and all(torch.equal(a, b) for a, b in zip(got, grads))


def test_gradient_against_differences(sb):
    x, dy, gamma, beta = draw(8, (2, 30, 24), "fp32")
    y, stats = sb.group_norm(x, 4, gamma, beta, activation="silu", return_stats=True)
    grads = [f64(t) for t in sb.group_norm_backward(dy, x, 4, stats, gamma, beta, activation="silu")]
    gen = np.random.default_rng(9)
    step = 1e-5
    for i, d in enumerate(grads):
        way = gen.standard_normal(d.shape)
        loss = []
        for sign in (1, -1):
            p = [f64(x), f64(gamma), f64(beta)]
            p[i] = p[i] + sign * step * way
            loss.append((ref.group_norm(p[0], 4, p[1], p[2], EPS, True)[0] * f64(dy)).sum())
        # the differences' own error is step^2 of the third derivative, the gradient's some
        # CHAIN U of the sum of its terms' magnitudes
        assert abs((loss[0] - loss[1]) / (2 * step) - (d * way).sum()) <= 2e-5 * np.abs(d * way).sum()


def test_no_positions(sb):
    x = torch.empty(2, 0, 8, device="cuda")
    y, stats = sb.group_norm(x, 2, return_stats=True)
    assert y.shape == x.shape
    gamma = torch.ones(8, device="cuda")
    dx, dgamma, dbeta = sb.group_norm_backward(x, x, 2, stats, gamma)
    assert dx.shape == x.shape and not dgamma.any() and not dbeta.any()
    assert sb.group_norm(torch.empty(0, 4, 8, device="cuda"), 2).shape == (0, 4, 8)


@pytest.mark.parametrize("dtype", DT)
def test_same_bits_every_time(sb, dtype):
    x, dy, gamma, beta = draw(10, (2, 700, 320), dtype)
    y, stats = sb.group_norm(x, 32, gamma, beta, activation="silu", return_stats=True)
    grads = sb.group_norm_backward(dy, x, 32, stats, gamma, beta, activation="silu")
    for _ in range(3):
        again = sb.group_norm(x, 32, gamma, beta, activation="silu", return_stats=True)
        assert torch.equal(again[0], y) and torch.equal(again[1], stats)
        more = sb.group_norm_backward(dy, x, 32, stats, gamma, beta, activation="silu")
        assert all(torch.equal(a, b) for a, b in zip(more, grads))


@pytest.mark.parametrize("shape", [(1, 16, 64), (2, 900, 320)], ids=str)
def test_prepared_calls_in_a_graph(sb, shape):
    x, dy, gamma, beta = draw(11, shape, "bf16")
    forward = sb.GroupNorm(x, 32, gamma, beta, activation="silu", return_stats=True)
    forward()
    back = sb.GroupNormBackward(dy, x, 32, forward.stats, gamma, beta, activation="silu")
    back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
        back()
    for turn in range(4):
        fresh = draw(20 + turn, shape, "bf16")
        for t, f in zip((x, dy, gamma, beta), fresh):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        y, stats = sb.group_norm(fresh[0], 32, *fresh[2:], activation="silu", return_stats=True)
        assert torch.equal(forward.out, y) and torch.equal(forward.stats, stats)
        for a, b in zip(back.out, sb.group_norm_backward(fresh[1], fresh[0], 32, stats, *fresh[2:], activation="silu")):
            assert torch.equal(a, b)


def test_writes_raise_the_version(sb):
    x, dy, gamma, beta = draw(12, (1, 8, 32), "fp32")
    out, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(1, 4, 3, device="cuda")
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    sb.group_norm(x, 4, stats=stats)
    for what, call in ((out, lambda: sb.group_norm(x, 4, out=out)), (stats, lambda: sb.group_norm(x, 4, stats=stats)),
                       (out, sb.GroupNorm(x, 4, out=out)), (dx, lambda: sb.group_norm_backward(dy, x, 4, stats, dx=dx)),
                       (dgamma, lambda: sb.group_norm_backward(dy, x, 4, stats, dgamma=dgamma)),
                       (dbeta, sb.GroupNormBackward(dy, x, 4, stats, dbeta=dbeta))):
        before, read = what._version, [t._version for t in (x, dy, gamma, beta)]
        call()
        assert what._version > before and [t._version for t in (x, dy, gamma, beta)] == read


def test_refusals(sb):
    x, dy, gamma, beta = draw(13, (2, 6, 6, 32), "fp16", "same")
    _, stats = sb.group_norm(x, 4, return_stats=True)
    bad = [
        (TypeError, lambda: sb.group_norm(x.cpu(), 4)), (TypeError, lambda: sb.group_norm(x.double(), 4)),
        (ValueError, lambda: sb.group_norm(x[0, 0, 0], 4)), (ValueError, lambda: sb.group_norm(x.permute(0, 3, 1, 2), 2)),
        (ValueError, lambda: sb.group_norm(x[:, :3, :3], 4, out=torch.empty_like(x))),
        (ValueError, lambda: sb.group_norm(x[:, ::2, :3], 4)), (ValueError, lambda: sb.group_norm(x, 4, activation="tanh")),
        (ValueError, lambda: sb.group_norm(x, 4, gamma[:16])), (ValueError, lambda: sb.group_norm(x, 4, gamma, beta.float())),
        (ValueError, lambda: sb.group_norm(x, 4, stats=stats[:1])), (sb.SeamBlendError, lambda: sb.group_norm(x, 5)),
        (sb.SeamBlendError, lambda: sb.group_norm(x, 0)), (sb.SeamBlendError, lambda: sb.group_norm(x, 4, eps=-1.0)),
        (sb.SeamBlendError, lambda: sb.group_norm(x[:, 1:], 4, out=x[:, :-1])),
        (ValueError, lambda: sb.group_norm_backward(dy[:1], x, 4, stats)),
        (ValueError, lambda: sb.group_norm_backward(dy, x, 4, stats.half())),
        (sb.SeamBlendError, lambda: sb.group_norm_backward(dy[:, 1:], x[:, 1:], 4, stats, dx=x[:, :-1])),
        (ValueError, lambda: sb.group_norm(x, 4, workspace=torch.empty(8, dtype=torch.uint8))),
        (sb.SeamBlendError, lambda: sb.group_norm(x, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k} was not refused")
