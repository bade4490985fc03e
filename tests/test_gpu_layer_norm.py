"""Layer norm, forward and backward, against its 64-bit definition."""
from __future__ import annotations

import sys

import numpy as np
import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def draw(shape, dtype, seed, mean=0.0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread + mean).to(dtype).cuda()


def weights(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda(), (0.3 * torch.randn(d, generator=g)).to(dtype).cuda()


def check(sb, x, dy, gamma, beta, eps=EPS, what=""):
    _say(f"[layer norm] {what} {tuple(x.shape)} {x.stride()} {x.dtype} {None if gamma is None else gamma.dtype}")
    w = None if gamma is None else ref.f64(gamma)
    b = None if beta is None else ref.f64(beta)
    y = sb.layer_norm(x, gamma, beta, eps=eps)
    assert y.dtype == x.dtype
    want, tol = ref.layer_norm(ref.f64(x), w, b, eps)
    ref.assert_near(y, want, tol, f"{what} y")
    dx, dgamma, dbeta = sb.layer_norm_backward(dy, x, gamma, eps=eps, weight_grads=True)
    assert dx.dtype == x.dtype and dgamma.dtype == dbeta.dtype == (F32 if gamma is None else gamma.dtype)
    wants, tols = ref.layer_norm_backward(ref.f64(dy), ref.f64(x), w, eps)
    for got, want, tol, name in zip((dx, dgamma, dbeta), wants, tols, ("dx", "dgamma", "dbeta")):
        ref.assert_near(got, want, tol, f"{what} {name}")
    alone, none_g, none_b = sb.layer_norm_backward(dy, x, gamma, eps=eps, weight_grads=False)
    assert none_g is None and none_b is None
    assert torch.equal(alone, dx)


# one element to rows past every register path, whole vectors and odd ends
WIDTHS = [1, 2, 3, 7, 8, 16, 31, 40, 64, 72, 127, 128, 255, 264, 500, 512, 768, 1000, 1153, 1536, 2048, 2056, 4096,
          5000, 8192, 8200, 16384, 16392, 20001, 33000, 70000]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("d", WIDTHS)
def test_widths(sb, d, dtype):
    rows = 37 if d <= 2048 else 5
    x, dy = draw((rows, d), dtype, d), draw((rows, d), dtype, d + 1)
    wt = F32 if d % 3 else dtype
    check(sb, x, dy, *weights(d, wt, d + 2), what=f"d={d}")


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 16, 17, 63, 64, 65, 128, 129, 257, 1031, 4099])
@pytest.mark.parametrize("d", [48, 320, 1280])
def test_row_counts(sb, rows, d):
    check(sb, draw((rows, d), BF16, rows), draw((rows, d), BF16, rows + 1), *weights(d, F32, 5), what=f"rows={rows}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("given", ["none", "gamma", "beta"])
def test_weights_given_or_not(sb, dtype, given):
    x, dy = draw((9, 136), dtype, 1), draw((9, 136), dtype, 2)
    gamma, beta = weights(136, dtype, 3)
    check(sb, x, dy, gamma if given == "gamma" else None, beta if given == "beta" else None, what=given)


@pytest.mark.parametrize("d", [64, 100, 1536, 9001, 50000])
def test_mean_large_against_the_spread(sb, d):
    x = draw((6, d), F32, d, mean=3000.0)
    check(sb, x, draw((6, d), F32, d + 1), *weights(d, F32, 3), what="mean 3000")


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("d", [65536, 300001])
def test_few_long_rows(sb, rows, d):
    check(sb, draw((rows, d), BF16, d), draw((rows, d), BF16, d + 1), *weights(d, F32, 3), what="long")
    check(sb, draw((rows, d), F32, d, mean=3000.0), draw((rows, d), F32, d + 1), None, None, what="long, mean 3000")


def test_loud_feature_first(sb):
    x = draw((8, 512), F32, 1)
    x[:, 0] = 3e4
    check(sb, x, draw((8, 512), F32, 2), *weights(512, F32, 3), what="loud")


def test_constant_rows_give_beta_and_no_gradient_through_the_spread(sb):
    x = torch.full((5, 96), 2.5, device="cuda")
    gamma, beta = weights(96, F32, 1)
    # what is left of x - mean is a rounding error of a rounding error, times 1000
    y = sb.layer_norm(x, gamma, beta, eps=EPS)
    assert torch.allclose(y, beta.expand(5, 96), rtol=2.0 ** -22, atol=1e-8)
    check(sb, x, draw((5, 96), F32, 2), gamma, beta, what="constant")


@pytest.mark.parametrize("d", [24, 200, 1536, 9000, 40000])
def test_nan_and_infinity_stay_in_their_row(sb, d):
    x, dy = draw((7, d), F32, 1), draw((7, d), F32, 2)
    clean, clean_dx, _ = sb.layer_norm(x), *sb.layer_norm_backward(dy, x)[:2]
    bad = x.clone()
    bad[2, d // 2], bad[5, 0] = float("nan"), float("inf")
    y, (dx, _, _) = sb.layer_norm(bad), sb.layer_norm_backward(dy, bad)
    for row in range(7):
        if row in (2, 5):
            assert torch.isnan(y[row]).all() and torch.isnan(dx[row]).all()
        else:
            assert torch.equal(y[row], clean[row]) and torch.equal(dx[row], clean_dx[row])


@pytest.mark.parametrize("d", [64, 128, 136])
def test_views_of_a_packed_projection(sb, d):
    packed = draw((11, 3, 5, d), BF16, 1)
    before = packed.clone()
    for part in range(3):
        x = packed[:, part]
        check(sb, x, draw((11, 5, d), BF16, part), *weights(d, BF16, 2), what=f"part {part}")
    assert torch.equal(packed, before)
    # out into another part of the same projection, and in place
    y = sb.layer_norm(packed[:, 0], out=packed[:, 1])
    assert torch.equal(y, sb.layer_norm(before[:, 0]))
    assert torch.equal(packed[:, 0], before[:, 0]) and torch.equal(packed[:, 2], before[:, 2])
    sb.layer_norm(packed[:, 2], out=packed[:, 2])
    assert torch.equal(packed[:, 2], sb.layer_norm(before[:, 2].contiguous()))


def test_three_axes_batch_slices_and_broadcast_rows(sb):
    whole = draw((4, 9, 96), F16, 1)
    x = whole[:, 2:7]
    check(sb, x, draw((4, 9, 96), F16, 2)[:, 1:6], *weights(96, F16, 3), what="slice")
    row = draw((1, 96), F16, 4).expand(6, 96)
    check(sb, row, draw((6, 96), F16, 5), *weights(96, F16, 3), what="broadcast")


@pytest.mark.parametrize("d", [128, 1001])
def test_offsets_past_32_bits(sb, d):
    far = torch.empty((1 << 31) + 4096, dtype=BF16, device="cuda")  # rows 2^30 elements apart
    x = far.as_strided((3, d), (1 << 30, 1))
    x.copy_(draw((3, d), BF16, 1))
    near, dy = x.clone(), draw((3, d), BF16, 2)
    want = [sb.layer_norm(near), *sb.layer_norm_backward(dy, near, weight_grads=True)]
    got = [sb.layer_norm(x), *sb.layer_norm_backward(dy, x, weight_grads=True)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    sb.layer_norm(x, out=x)
    assert torch.equal(x, want[0])


@pytest.mark.parametrize("offset", [1, 2, 3, 5])
@pytest.mark.parametrize("d", [129, 1027])
def test_odd_offsets(sb, offset, d):
    base, grad = draw((6 * d + 8,), BF16, 1), draw((6 * d + 8,), BF16, 2)
    x, dy = base[offset:offset + 6 * d].view(6, d), grad[8 - offset:8 - offset + 6 * d].view(6, d)
    check(sb, x, dy, *weights(d, BF16, 3), what=f"offset {offset}")
    # the elements around the output stay as they are
    out = torch.full((6 * d + 8,), 7.0, dtype=BF16, device="cuda")
    sb.layer_norm(x, out=out[offset:offset + 6 * d].view(6, d))
    assert (out[:offset] == 7).all() and (out[offset + 6 * d:] == 7).all()


@pytest.mark.parametrize("d", [40, 777, 9001, 40000])
def test_gradient_in_place(sb, d):
    x, dy = draw((5, d), F32, 1), draw((5, d), F32, 2)
    gamma, _ = weights(d, F32, 3)
    want = sb.layer_norm_backward(dy, x, gamma)
    for alias in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        got = sb.layer_norm_backward(a, b, gamma, dx=a if alias == "dy" else b)
        assert all(torch.equal(g, w) for g, w in zip(got, want)), alias


def test_no_rows(sb):
    x = torch.empty(0, 3, 64, dtype=BF16, device="cuda")
    gamma, beta = weights(64, F32, 1)
    assert sb.layer_norm(x, gamma, beta).shape == x.shape
    dx, dgamma, dbeta = sb.layer_norm_backward(x, x, gamma)
    assert dx.shape == x.shape and not dgamma.any() and not dbeta.any()


@pytest.mark.parametrize("d", [33, 600])
def test_gradient_against_differences(sb, d):
    """dx, dgamma and dbeta along random directions against central differences of
    the 64-bit definition.  Step 1e-5: the differences are off by about 1e-10
    (third derivative) and 1e-11 (rounding) of the terms' size, far below the
    kernels' own bounds."""
    rng = np.random.default_rng(d)
    x, dy = draw((4, d), F32, 1), draw((4, d), F32, 2)
    gamma, beta = weights(d, F32, 3)
    got = sb.layer_norm_backward(dy, x, gamma)
    _, tols = ref.layer_norm_backward(ref.f64(dy), ref.f64(x), ref.f64(gamma), EPS)
    at = [ref.f64(x), ref.f64(gamma), ref.f64(beta)]
    loss = lambda p: (ref.layer_norm(*p, EPS)[0] * ref.f64(dy)).sum()  # noqa: E731
    for which in range(3):
        v = rng.standard_normal(at[which].shape)
        up, down = list(at), list(at)
        up[which], down[which] = at[which] + 1e-5 * v, at[which] - 1e-5 * v
        slope = (loss(up) - loss(down)) / 2e-5
        mine = (ref.f64(got[which]) * v).sum()
        allowed = (tols[which] * np.abs(v)).sum() + 1e-7 * np.abs(ref.f64(got[which]) * v).sum()
        assert abs(mine - slope) <= allowed, f"parameter {which}: {mine} against {slope}, allowed {allowed}"


def test_same_bits_every_time_and_on_another_stream(sb):
    x, dy = draw((3001, 320), BF16, 1), draw((3001, 320), BF16, 2)
    gamma, beta = weights(320, F32, 3)
    first = [sb.layer_norm(x, gamma, beta), *sb.layer_norm_backward(dy, x, gamma)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [sb.layer_norm(x, gamma, beta), *sb.layer_norm_backward(dy, x, gamma)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_prepared_calls_in_a_graph(sb):
    x, dy = draw((130, 384), BF16, 1), draw((130, 384), BF16, 2)
    gamma, beta = weights(384, F32, 3)
    forward, backward = sb.LayerNorm(x, gamma, beta), sb.LayerNormBackward(dy, x, gamma)
    forward(), backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward(), backward()
    for seed in (11, 12, 13):
        x.copy_(draw((130, 384), BF16, seed))
        want = [sb.layer_norm(x, gamma, beta), *sb.layer_norm_backward(dy, x, gamma)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([forward.out, *backward.out], want))


def test_refusals(sb):
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(TypeError):
        sb.layer_norm(x.cpu())
    with pytest.raises(TypeError):
        sb.layer_norm(x.double())
    with pytest.raises(ValueError):
        sb.layer_norm(x.t())  # last axis not contiguous
    with pytest.raises(ValueError):
        sb.layer_norm(torch.zeros(2, 3, 4, 5, 8, device="cuda")[:, ::2, :, ::2])  # more than two strided axes
    with pytest.raises(ValueError):
        sb.layer_norm(x, gamma=torch.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        sb.layer_norm(x, gamma=torch.ones(8, device="cuda", dtype=F16))
    with pytest.raises(ValueError):
        sb.layer_norm(x, gamma=torch.ones(8))
    with pytest.raises(ValueError):
        sb.layer_norm(x, out=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        sb.layer_norm_backward(torch.zeros(3, 8, device="cuda"), x)
    flat = torch.zeros(64, device="cuda")
    with pytest.raises(sb.SeamBlendError) as e:
        sb.layer_norm(flat[:32].view(4, 8), out=flat[4:36].view(4, 8))
    assert e.value.code == -1 and "overlaps" in str(e.value)
    with pytest.raises(sb.SeamBlendError):
        sb.layer_norm(x, out=torch.zeros(1, 8, device="cuda").expand(4, 8))
    with pytest.raises(sb.SeamBlendError):
        sb.layer_norm(x, eps=-1.0)
    with pytest.raises(sb.SeamBlendError) as e:
        sb.layer_norm_backward(x, x, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -3
