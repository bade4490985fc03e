"""The transformer operators at the sizes where they take another way: outputs
that pass the caches, longer chunks of a clip, more rows, tokens or steps than
one grid or launch holds.  Compared on the GPU with the definitions in 64 bits,
in pieces, under the bounds of transformer_ref."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6
LAST_LEVEL = 256 << 20  # bytes of the memory-side cache
#: binary digits after the first, and the least exponent, of the 16-bit types
DIGITS = {F16: (10, -14), BF16: (7, -126)}


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _say(*a):
    print("[large]", *a, file=sys.stderr, flush=True)


def normal(shape, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for piece in out.flatten().split(1 << 26):
        piece.copy_(torch.randn(piece.shape, generator=gen, device="cuda"))
    return out


def assert_near(got, want, tol, what):
    """got within tol of want and the rounding of its type (the half step of the
    next binade where want may fall into it; fp32's is counted in tol)."""
    off = (got.double() - want).abs_() - tol
    if got.dtype != F32:
        digits, least = DIGITS[got.dtype]
        size = (want.abs() + tol) * (1 + 2.0 ** -9)
        exponent = torch.floor(torch.log2(size.clamp_min(2.0 ** least)))
        off -= torch.exp2(exponent - digits - 1)
    worst = off.max().item()
    assert worst <= 0, f"{what}: {int((off > 0).sum())} of {got.numel()} off, by up to {worst}"


def weights(d, dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda: torch.randn(d, generator=gen, device="cuda")  # noqa: E731
    return (1 + 0.3 * draw()).to(dtype), (0.3 * draw()).to(dtype)


def check_forward(y, x, gamma, beta, what):
    d = x.shape[-1]
    for k in range(0, x.shape[0], step := max(1, (1 << 25) // d)):
        v = x[k:k + step].double()
        m = v.mean(-1, keepdim=True)
        h = (v - m) / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + EPS)
        want = h * gamma.double() + beta.double()
        tol = ref.chain(d) * ref.U * ((1 + h.abs()) * gamma.double().abs() + want.abs())
        assert_near(y[k:k + step], want, tol, f"{what} y from row {k}")


def check_backward(got, dy, x, gamma, what):
    dx, dgamma, dbeta = got
    rows, d = x.shape
    c = ref.chain(d) * ref.U
    sums = [torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(4)]
    for k in range(0, rows, step := max(1, (1 << 25) // d)):
        v, g0 = x[k:k + step].double(), dy[k:k + step].double()
        m = v.mean(-1, keepdim=True)
        r = 1 / torch.sqrt(((v - m) ** 2).mean(-1, keepdim=True) + EPS)
        h = (v - m) * r
        g = g0 * gamma.double()
        ah, ag = 1 + h.abs(), g.abs()
        want = r * (g - g.mean(-1, keepdim=True) - h * (g * h).mean(-1, keepdim=True))
        tol = 2 * c * r * (ag + ag.mean(-1, keepdim=True) + ah * (ag * ah).mean(-1, keepdim=True))
        assert_near(dx[k:k + step], want, tol, f"{what} dx from row {k}")
        for s, term in zip(sums, (g0 * h, g0, g0.abs() * ah, g0.abs())):
            s += term.sum(0)
    assert_near(dgamma, sums[0], (c + rows * ref.U) * sums[2], f"{what} dgamma")
    assert_near(dbeta, sums[1], (rows + 8) * ref.U * sums[3], f"{what} dbeta")


# rows of every layout, whole vectors: 64 to 4096 of them
@pytest.mark.parametrize("dtype,d", [(BF16, 512), (F16, 1024), (BF16, 1536), (F16, 2048), (F32, 1024), (BF16, 2560),
                                     (BF16, 4096), (F16, 6144), (F32, 4096), (BF16, 8192), (BF16, 16384),
                                     (F16, 24576), (F32, 16384)])
def test_layer_norm_outputs_past_the_caches(sb, dtype, d):
    rows = LAST_LEVEL // (d * (4 if dtype == F32 else 2)) + 1
    _say("layer norm", rows, d, dtype)
    x, dy = normal((rows, d), dtype, d), normal((rows, d), dtype, d + 1)
    gamma, beta = weights(d, F32 if d % 1024 else dtype, d + 2)
    y = sb.layer_norm(x, gamma, beta, eps=EPS)
    check_forward(y, x, gamma, beta, f"{dtype} {d}")
    y.copy_(x)
    assert torch.equal(sb.layer_norm(y, gamma, beta, eps=EPS, out=y)[:7], sb.layer_norm(x[:7], gamma, beta, eps=EPS))
    check_forward(y, x, gamma, beta, f"{dtype} {d} in place")
    got = sb.layer_norm_backward(dy, x, gamma, eps=EPS)
    check_backward(got, dy, x, gamma, f"{dtype} {d}")
    place = dy.clone()
    again = sb.layer_norm_backward(place, x, gamma, eps=EPS, dx=place)
    assert all(torch.equal(a, b) for a, b in zip(again, got))


@pytest.mark.parametrize("rows,d", [(1100, 33000), (65600, 32776)])
def test_more_long_rows_than_a_grid_is_high(sb, rows, d):
    _say("long rows", rows, d)
    x = normal((rows, d), BF16, 1)
    gamma, beta = weights(d, F32, 2)
    check_forward(sb.layer_norm(x, gamma, beta, eps=EPS), x, gamma, beta, f"{rows} x {d}")


@pytest.mark.parametrize("rows,d", [(2100, 16392), (65600, 16392)])
def test_more_long_rows_than_a_grid_is_high_backward(sb, rows, d):
    _say("long rows, backward", rows, d)
    x, dy = normal((rows, d), BF16, 1), normal((rows, d), BF16, 2)
    gamma, _ = weights(d, F32, 3)
    check_backward(sb.layer_norm_backward(dy, x, gamma, eps=EPS), dy, x, gamma, f"{rows} x {d}")


def test_as_many_rows_as_there_can_be(sb):
    """2^31 - 1 rows of 2: more blocks of 128 than a grid has.  1024 different
    rows, over and over."""
    rows, period = (1 << 31) - 1, 1024
    _say("layer norm", rows, 2)
    some = normal((period, 2), BF16, 1)
    want = sb.layer_norm(some, eps=EPS)
    ones = torch.ones(2, device="cuda")
    check_forward(want, some, ones, 0 * ones, "1024 rows")
    x = some.repeat((rows + 1) // period, 1)[:rows]
    sb.layer_norm(x, eps=EPS, out=x)
    whole = rows // period * period
    for piece in x[:whole].view(-1, 2 * period).split(1 << 16):
        assert (piece == want.flatten()).all()
    assert torch.equal(x[whole:], want[:rows - whole])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_of_more_steps_than_a_launch_takes(sb, interleaved):
    """2^30 tokens and a few of one query and one key head of 2: the last 3073 of
    them in a launch of their own.  1024 different tokens, over and over."""
    batch, length = (1 << 20) + 3, 1024
    _say("rotary", batch, length, interleaved)
    f, _ = sb.rotary_frequencies(2)
    positions = torch.arange(length, device="cuda")
    q, k = normal((1, length, 1, 2), BF16, 1), normal((1, length, 1, 2), BF16, 2)
    want = sb.rotary(q, positions, f, k=k, interleaved=interleaved)
    for x, y in zip((q, k), want):
        turned, tol = ref.rotary(ref.f64(x), positions.cpu().numpy()[None, None], f.cpu().numpy(), (1,), interleaved, 1.0)
        ref.assert_near(y, turned, tol, "1024 tokens")
    q, k = q.repeat(batch, 1, 1, 1), k.repeat(batch, 1, 1, 1)
    sb.rotary(q, positions, f, k=k, interleaved=interleaved, out=q, k_out=k)
    for got, w in zip((q, k), want):
        for piece in got.view(batch, 2 * length).split(1 << 16):
            assert (piece == w.flatten()).all()


def check_clip(sb, grads, outs, max_norm, what):
    """outs: None for in place.  (norm's sum is 64-bit: off by its one rounding.)"""
    _say("clip", what, len(grads), "tensors,", sum(g.numel() for g in grads), "elements")
    before = [g.clone() for g in grads]
    norm = math.sqrt(sum(g.double().square().sum().item() for g in before))
    got = sb.grad_norm_clip(grads, max_norm, eps=EPS, out=outs).item()
    assert abs(got - norm) <= 2 * ref.U * norm, what
    by = min(1.0, max_norm / (norm + EPS))
    for g, b, o in zip(grads, before, grads if outs is None else outs):
        assert outs is None or torch.equal(g, b), f"{what}: a gradient changed"
        want = b.double() * by
        assert_near(o, want, 4 * ref.U * want.abs() + 2.0 ** -149, what)


def tensors(bucket, offset):
    """Views of a bucket from an odd offset on: a few large ones, odd lengths,
    neighbours, the last few elements left."""
    n = bucket.numel() - offset - 9
    sizes = [1, n // 2 - 3, 7, n // 3, 4099]
    return list(bucket[offset:offset + n].split(sizes + [n - sum(sizes)]))


# elements: chunks of more than 8192 (over 2^25), and with 256 MiB or more moved
@pytest.mark.parametrize("dtype,out,n", [(BF16, F32, 47_000_001), (F16, F32, 47_000_001), (F32, F32, 36_000_001),
                                         (F16, F16, 70_000_003), (BF16, BF16, 70_000_003), (BF16, BF16, 40_000_001),
                                         (F32, None, 36_000_001), (F32, None, 70_000_003), (BF16, None, 36_000_001),
                                         (BF16, None, 140_000_003), (F16, None, 140_000_003), (F32, F32, 1_000_001)])
@pytest.mark.parametrize("offset", [0, 3])
def test_large_clips(sb, dtype, out, n, offset):
    bucket = normal((n,), dtype, n)
    grads = tensors(bucket, offset)
    ends = bucket[:offset].clone(), bucket[n - 9:].clone()
    outs = None
    if out is not None:
        to = torch.full((n + 1,), 7.0, dtype=out, device="cuda")
        outs = tensors(to[:n], offset)
    check_clip(sb, grads, outs, 0.3 * math.sqrt(n), f"{dtype} to {out} from {offset}")
    assert torch.equal(bucket[:offset], ends[0]) and torch.equal(bucket[n - 9:], ends[1])
    if out is not None:
        assert (to[:offset] == 7).all() and (to[n - 9:] == 7).all()


def test_large_clip_below_the_bound(sb):
    grads = tensors(normal((70_000_003,), F32, 1), 1)
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    assert sb.grad_norm_clip(grads, 1e9).item() == sb.grad_norm_clip(grads, 1e9, out=outs).item()
    assert all(torch.equal(g, b) and torch.equal(o, b) for g, b, o in zip(grads, before, outs))
