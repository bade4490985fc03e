"""The gradient norm over many tensors, and clipping, against the definition."""
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


def draw(shapes, dtypes, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * spread).to(dtypes[k % len(dtypes)]).cuda() for k, s in enumerate(shapes)]


def check(sb, grads, max_norm, out_dtype=None, what=""):
    print(f"[clip] {what} {len(grads)} tensors, {sum(g.numel() for g in grads)} elements", file=sys.stderr, flush=True)
    host = [ref.f64(g) for g in grads]
    norm, tol, want, tols = ref.clip(host, max_norm, EPS)
    only = sb.grad_norm(grads)
    assert only.shape == () and only.dtype == F32
    assert abs(only.item() - norm) <= tol, f"{what}: norm {only.item()}, expected {norm}"
    outs = [torch.full(g.shape, 7.0, dtype=out_dtype or g.dtype, device="cuda") for g in grads]
    before = [g.clone() for g in grads]
    got = sb.grad_norm_clip(grads, max_norm, eps=EPS, out=outs)
    assert torch.equal(got, only)
    assert all(torch.equal(a, b) for a, b in zip(grads, before)), "inputs changed"
    for o, w, t in zip(outs, want, tols):
        ref.assert_near(o, w, t, what)
    place = [g.clone() for g in grads]
    assert torch.equal(sb.grad_norm_clip(place, max_norm, eps=EPS), only)
    for p, w, t in zip(place, want, tols):
        ref.assert_near(p, w, t, f"{what} in place")


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 16383, 16384, 16385, 100003])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_lengths(sb, n, dtype):
    check(sb, draw([(n,)], [dtype], n), 0.5, what=f"n={n}")


@pytest.mark.parametrize("out_dtype", [None, F32])
def test_mixed_types_shapes_and_empty_tensors(sb, out_dtype):
    shapes = [(3, 5), (0,), (1,), (17, 33, 2), (), (40000,), (2, 0, 4), (129,), (64, 64)]
    check(sb, draw(shapes, [F32, BF16, F16, BF16], 1), 3.0, out_dtype, "mixed")


@pytest.mark.parametrize("count", [127, 128, 129, 300, 1000])
def test_more_tensors_than_a_launch_takes(sb, count):
    check(sb, draw([(1 + 37 * k % 101,) for k in range(count)], [F32, BF16], count), 1.0, what="many")


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1e9, float("inf")])
def test_bounds(sb, max_norm):
    grads = draw([(1000,), (33, 3)], [F32], 1)
    check(sb, grads, max_norm, what=f"bound {max_norm}")
    if max_norm > 1e3:  # below the bound the bits stay
        before = [g.clone() for g in grads]
        sb.grad_norm_clip(grads, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))


@pytest.mark.parametrize("spread", [1e-30, 1e-22, 1e18, 1e30])
def test_squares_neither_overflow_nor_vanish(sb, spread):
    check(sb, draw([(5000,), (3,)], [F32, BF16], 1, spread), spread, what=f"spread {spread}")


def test_nothing_but_zeros_and_nothing_at_all(sb):
    zeros = [torch.zeros(100, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]
    assert sb.grad_norm_clip(zeros, 1.0).item() == 0 and not any(z.any() for z in zeros)
    empty = [torch.empty(0, device="cuda")]
    assert sb.grad_norm_clip(empty, 1.0).item() == 0 and sb.grad_norm(empty).item() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_norms_that_are_not_finite(sb, bad):
    grads = draw([(300,), (20,)], [F32], 1)
    grads[1][7] = bad
    norm = sb.grad_norm_clip(grads, 1.0)
    if bad != bad:
        assert torch.isnan(norm) and all(torch.isnan(g).all() for g in grads)
    else:
        assert torch.isposinf(norm) and torch.isnan(grads[1][7])
        grads[1][7] = 0
        assert not any(g.any() for g in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_views_of_a_bucket_at_odd_offsets(sb, dtype):
    bucket = draw([(4099,)], [dtype], 1)[0]
    sizes = [1, 5, 1023, 7, 2000, 1063]
    check(sb, list(bucket.split(sizes)), 2.0, what="bucket")
    out = torch.full((4110,), 7.0, device="cuda")
    sb.grad_norm_clip(list(bucket.split(sizes)), 2.0, out=list(out[3:4102].split(sizes)))
    assert (out[:3] == 7).all() and (out[4102:] == 7).all()


def test_dense_tensors_in_another_order(sb):
    g = draw([(4, 6, 5, 3)], [F32], 1)[0].to(memory_format=torch.channels_last)
    assert not g.is_contiguous()
    norm, tol, want, tols = ref.clip([ref.f64(g)], 1.0, EPS)
    assert abs(sb.grad_norm_clip([g], 1.0).item() - norm) <= tol
    ref.assert_near(g, want[0], tols[0], "channels last")


def test_same_bits_every_time_in_a_graph_and_on_another_stream(sb):
    grads = draw([(70001,), (333,), (5, 5)], [BF16, F32], 1)
    outs = [torch.empty(g.shape, device="cuda") for g in grads]
    plan = sb.GradNormClip(grads, 0.7, out=outs)
    first = plan().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for step in range(3):
        for g in grads:
            g.mul_(1.5)
        want = [torch.empty(g.shape, device="cuda") for g in grads]
        norm = sb.grad_norm_clip(grads, 0.7, out=want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.norm, norm) and not torch.equal(norm, first)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = sb.grad_norm(grads)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, norm)


def test_refusals(sb):
    g = torch.zeros(4, 6, device="cuda")
    with pytest.raises(ValueError):
        sb.grad_norm([])
    with pytest.raises(TypeError):
        sb.grad_norm([g.cpu()])
    with pytest.raises(TypeError):
        sb.grad_norm([g, g.double()])
    with pytest.raises(ValueError):
        sb.grad_norm([g[:, ::2]])
    with pytest.raises(ValueError):
        sb.grad_norm([g[:1].expand(4, 6)])
    with pytest.raises(ValueError):
        sb.grad_norm_clip([g], 1.0, out=[])
    with pytest.raises(ValueError):
        sb.grad_norm_clip([g], 1.0, out=[torch.zeros(6, 4, device="cuda")])
    with pytest.raises(ValueError):
        sb.grad_norm_clip([g], 1.0, out=[g.half()])
    with pytest.raises(ValueError):
        sb.grad_norm_clip([g, g], 1.0)
    with pytest.raises(ValueError):
        sb.grad_norm_clip([g, g.clone()], 1.0, out=[g, g])
    assert sb.grad_norm([g, g]).item() == 0  # nothing is written
    flat = torch.zeros(40, device="cuda")
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(max_norm=1.0, eps=-1.0)):
        with pytest.raises(sb.SeamBlendError):
            sb.grad_norm_clip([g], **bad)
    with pytest.raises(sb.SeamBlendError) as e:
        sb.grad_norm_clip([flat[:24]], 1.0, out=[flat[4:28]])
    assert e.value.code == -1 and "overlaps" in str(e.value)
