"""Rotary position embedding against its 64-bit definition."""
from __future__ import annotations

import math
import sys

import numpy as np
import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def draw(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def check(sb, q, k, positions, freqs, interleaved, sections=None, scale=1.0, what=""):
    print(f"[rotary] {what} {tuple(q.shape)} {None if k is None else tuple(k.shape)} {q.dtype} "
          f"pairs={freqs.numel()} inter={interleaved} {sections}", file=sys.stderr, flush=True)
    b, t = (q.shape[0], q.shape[1]) if q.dim() == 4 else (1, q.shape[0])
    p = positions if sections is not None else positions.unsqueeze(0)
    p = np.broadcast_to(p.cpu().numpy().reshape(p.shape[0], -1, t), (p.shape[0], b, t))
    parts = (freqs.numel(),) if sections is None else sections
    for call, transpose in ((sb.rotary, False), (sb.rotary_backward, True)):
        out = call(q, positions, freqs, k=k, interleaved=interleaved, sections=sections, scale=scale)
        for got, x in zip((out,) if k is None else out, (q, k)):
            assert got.dtype == x.dtype
            want, tol = ref.rotary(ref.f64(x).reshape(b, t, *x.shape[-2:]), p, freqs.cpu().numpy(), parts,
                                   interleaved, scale, transpose)
            ref.assert_near(got.reshape(want.shape), want, tol, f"{what} transpose={transpose}")


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,part", [(2, 2), (3, 2), (8, 8), (32, 32), (64, 64), (72, 50), (80, 40), (96, 96),
                                    (127, 126), (128, 128), (128, 6), (256, 256), (1000, 770)])
def test_head_shapes(sb, dtype, interleaved, d, part):
    f, _ = sb.rotary_frequencies(part)
    q, k = draw((2, 5, 3, d), dtype, d), draw((2, 5, 1, d), dtype, d + 1)
    positions = torch.tensor([[0, 1, 2, 3, 4], [100, 7, 5, 99999, 12]], device="cuda")
    check(sb, q, k, positions, f, interleaved, what=f"d={d} part={part}")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,part", [(8192, 8192), (8191, 8190), (5000, 4096)])
def test_longest_heads(sb, interleaved, d, part):
    f, _ = sb.rotary_frequencies(part)
    check(sb, draw((3, 1, d), BF16, 1), draw((3, 2, d), BF16, 2), torch.tensor([0, 5, 70000], device="cuda"), f,
          interleaved, what="long heads")
    with pytest.raises(sb.SeamBlendError):
        sb.rotary(draw((1, 1, 8194), F32, 1), torch.zeros(1, dtype=torch.int64, device="cuda"), f)


@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (8, 2), (12, 12), (32, 8), (40, 40), (130, 2)])
@pytest.mark.parametrize("tokens", [1, 2, 33, 257])
def test_head_and_token_counts(sb, heads, tokens):
    f, _ = sb.rotary_frequencies(64)
    check(sb, draw((tokens, heads[0], 64), BF16, 1), draw((tokens, heads[1], 64), BF16, 2),
          torch.arange(tokens, device="cuda") + 17, f, tokens % 2 == 0, what="counts")


@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_far_and_negative_positions(sb, kind):
    f, _ = sb.rotary_frequencies(128)
    positions = torch.tensor([0, -1, -77777, 1 << 20, (1 << 20) + 1, (1 << 31) - 1, -(1 << 31)],
                             dtype=torch.int64, device="cuda").to(kind)
    check(sb, draw((7, 2, 128), F32, 1), None, positions, f, False, what="far")


def test_positions_past_32_bits(sb):
    f, _ = sb.rotary_frequencies(16)
    check(sb, draw((3, 2, 16), F32, 1), None, torch.tensor([1 << 33, (1 << 33) + 5, -(1 << 34)], device="cuda"), f, True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections", [(16, 8, 8), (11, 10, 11), (5, 27), (32,), (0, 16, 0, 16), (8, 8, 8, 8)])
def test_axes(sb, sections, interleaved):
    f, _ = sb.rotary_frequencies(64, sections=sections)
    frames, rows, cols = 3, 5, 7
    grid = torch.cartesian_prod(torch.arange(frames), torch.arange(rows), torch.arange(cols)).t()
    p = torch.cat((grid, grid[:1] * 9 + 1))[:len(sections)].contiguous().cuda()
    check(sb, draw((105, 4, 64), BF16, 1), draw((105, 2, 64), BF16, 2), p, f, interleaved, sections, what="axes")
    pb = torch.stack((p, p + 3), 1)  # [axes, B, T]
    check(sb, draw((2, 105, 4, 64), F16, 1), None, pb, f, interleaved, sections, what="axes, batch")


def test_broadcast_and_strided_positions(sb):
    f, _ = sb.rotary_frequencies(32)
    q = draw((3, 9, 2, 32), F32, 1)
    check(sb, q, None, torch.arange(9, device="cuda"), f, False, what="[T]")
    check(sb, q, None, torch.arange(9, device="cuda").expand(1, 9), f, False, what="[1, T]")
    check(sb, q, None, torch.arange(27, device="cuda").view(9, 3).t(), f, False, what="strided [B, T]")
    check(sb, q, None, torch.arange(18, device="cuda")[::2].expand(3, 9), f, False, what="expanded")


@pytest.mark.parametrize("interleaved", [False, True])
def test_views_in_place_and_between_views(sb, interleaved):
    f, _ = sb.rotary_frequencies(48)
    positions = torch.arange(6, device="cuda") * 31
    packed = draw((2, 6, 4 + 2 + 2, 64), BF16, 1)
    before = packed.clone()
    q, k = packed[:, :, :4], packed[:, :, 4:6]
    check(sb, q, k, positions, f, interleaved, what="packed")
    want_q, want_k = sb.rotary(q, positions, f, k=k, interleaved=interleaved)
    sb.rotary(q, positions, f, k=k, interleaved=interleaved, out=q, k_out=k)  # in place, both views of one buffer
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(packed[:, :, 6:], before[:, :, 6:])
    # heads before tokens
    q, k = draw((2, 4, 6, 64), F32, 2).transpose(1, 2), draw((2, 2, 6, 64), F32, 3).transpose(1, 2)
    check(sb, q, k, positions, f, interleaved, what="head-major")


def test_offsets_past_32_bits(sb):
    f, _ = sb.rotary_frequencies(64)
    far = torch.empty((1 << 31) + 4096, dtype=BF16, device="cuda")  # elements 2^30 and 2^31 bytes apart and more
    q = far.as_strided((3, 2, 64), (1 << 30, 64, 1))
    q.copy_(draw((3, 2, 64), BF16, 1))
    near = q.clone()
    positions = torch.tensor([5, 6, 7], device="cuda")
    want = sb.rotary(near, positions, f)
    assert torch.equal(sb.rotary(q, positions, f), want)
    sb.rotary(q, positions, f, out=q)
    assert torch.equal(q, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_odd_offsets_and_neighbours_untouched(sb, interleaved):
    f, _ = sb.rotary_frequencies(26)
    flat, out = draw((5 * 3 * 37 + 9,), BF16, 1), torch.full((5 * 3 * 37 + 9,), 7.0, dtype=BF16, device="cuda")
    for o in (1, 3, 4):
        q = flat[o:o + 555].view(5, 3, 37)
        check(sb, q, None, torch.arange(5, device="cuda"), f, interleaved, what=f"offset {o}")
        out.fill_(7.0)
        sb.rotary(q, torch.arange(5, device="cuda"), f, interleaved=interleaved, out=out[9 - o:564 - o].view(5, 3, 37))
        assert (out[:9 - o] == 7).all() and (out[564 - o:] == 7).all()


@pytest.mark.parametrize("scaling,more", [("linear", {}), ("base", {}), ("by_parts", {"original_length": 512})])
def test_frequencies(sb, scaling, more):
    f, scale = sb.rotary_frequencies(32, 10000.0, scaling, 8.0, **more)
    plain, one = sb.rotary_frequencies(32)
    assert one == 1.0 and f.dtype == torch.float64 and f.numel() == 16
    f, plain = f.cpu().numpy(), plain.cpu().numpy()
    assert np.allclose(plain, 10000.0 ** (-np.arange(16) / 16), rtol=1e-15)
    if scaling == "linear":
        assert np.array_equal(f, plain / 8) and scale == 1.0
    elif scaling == "base":
        assert f[0] == 1.0 and math.isclose(f[-1], plain[-1] / 8, rel_tol=1e-12) and scale == 1.0
    else:
        turns = 512 * plain / (2 * math.pi)
        assert np.array_equal(f[turns >= 32], plain[turns >= 32])
        assert np.array_equal(f[turns <= 1], plain[turns <= 1] / 8)
        mixed = (turns > 1) & (turns < 32)
        assert mixed.any() and (f[mixed] < plain[mixed]).all() and (f[mixed] > plain[mixed] / 8).all()
        assert math.isclose(scale, 0.1 * math.log(8) + 1)
    q = draw((4, 2, 32), F32, 1)
    fd = torch.from_numpy(f).cuda()
    check(sb, q, None, torch.arange(4, device="cuda") * 1000, fd, False, scale=scale, what=scaling)


def test_gradient_is_the_transpose(sb):
    """<dy, rotary(x)> == <rotary_backward(dy), x> up to the two calls' bounds, and
    against differences: the map is linear, so rotary(x + v) - rotary(x) is its
    directional derivative up to three roundings of its terms."""
    f, _ = sb.rotary_frequencies(40, sections=(7, 13))
    p = torch.arange(22, device="cuda").view(2, 11)
    x, v, dy = (draw((11, 3, 48), F32, s) for s in (1, 2, 3))
    args = dict(sections=(7, 13), scale=1.3, interleaved=True)
    y, dx = sb.rotary(x, p, f, **args), sb.rotary_backward(dy, p, f, **args)
    size = (1.3 * (np.abs(ref.f64(x)).max() + np.abs(ref.f64(v)).max()) * 2 * np.abs(ref.f64(dy))).sum()
    assert abs((ref.f64(y) * ref.f64(dy)).sum() - (ref.f64(x) * ref.f64(dx)).sum()) <= 24 * ref.U * size
    slope = ((ref.f64(sb.rotary(x + v, p, f, **args)) - ref.f64(y)) * ref.f64(dy)).sum()
    assert abs(slope - (ref.f64(dx) * ref.f64(v)).sum()) <= 48 * ref.U * size


def test_infinity_and_nan_stay_in_their_pair(sb):
    f, _ = sb.rotary_frequencies(16)
    x = draw((3, 2, 16), F32, 1)
    clean = sb.rotary(x, torch.arange(3, device="cuda"), f)
    x[1, 1, 3], x[2, 0, 5] = float("nan"), float("inf")
    y = sb.rotary(x, torch.arange(3, device="cuda"), f)
    touched = torch.zeros_like(x, dtype=torch.bool)
    touched[1, 1, [3, 11]] = touched[2, 0, [5, 13]] = True
    assert torch.equal(y[~touched], clean[~touched]) and not torch.isfinite(y[touched]).any()


def test_no_tokens(sb):
    f, _ = sb.rotary_frequencies(16)
    q = torch.empty(2, 0, 3, 16, device="cuda")
    assert sb.rotary(q, torch.empty(2, 0, dtype=torch.int64, device="cuda"), f).shape == q.shape


def test_prepared_call_in_a_graph_and_on_a_stream(sb):
    f, _ = sb.rotary_frequencies(64)
    q, k, p = draw((4, 1, 8, 64), BF16, 1), draw((4, 1, 2, 64), BF16, 2), torch.arange(4, device="cuda").view(4, 1)
    plan = sb.Rotary(q, p, f, k)
    plan()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for step in range(3):
        p += 100
        want = sb.rotary(q, p, f, k=k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out[0], want[0]) and torch.equal(plan.out[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = sb.rotary(q, p, f, k=k)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_refusals(sb):
    f, _ = sb.rotary_frequencies(16)
    q, p = torch.zeros(3, 2, 16, device="cuda"), torch.arange(3, device="cuda")
    with pytest.raises(TypeError):
        sb.rotary(q.cpu(), p, f)
    with pytest.raises(TypeError):
        sb.rotary(q.double(), p, f)
    with pytest.raises(ValueError):
        sb.rotary(q[0], p, f)
    with pytest.raises(ValueError):
        sb.rotary(q, p.float(), f)
    with pytest.raises(ValueError):
        sb.rotary(q, p[:2], f)
    with pytest.raises(ValueError):
        sb.rotary(q, p, f.float())
    with pytest.raises(ValueError):
        sb.rotary(q, p, f, k=torch.zeros(3, 2, 8, device="cuda"))
    with pytest.raises(ValueError):
        sb.rotary(q, p, f, sections=(4, 4))  # positions lack the axis
    with pytest.raises(sb.SeamBlendError):
        sb.rotary(q, torch.stack((p, p)), f, sections=(4, 5))
    with pytest.raises(sb.SeamBlendError):
        sb.rotary(q, p, torch.cat((f, f)))  # more pairs than the head holds
    with pytest.raises(sb.SeamBlendError):
        sb.rotary(q, p, f, scale=float("inf"))
    flat = torch.zeros(200, device="cuda")
    with pytest.raises(sb.SeamBlendError) as e:
        sb.rotary(flat[:96].view(3, 2, 16), p, f, out=flat[16:112].view(3, 2, 16))
    assert e.value.code == -1 and "overlaps" in str(e.value)
    with pytest.raises(sb.SeamBlendError):  # the key heads' output over the query heads
        sb.rotary(q, p, f, k=q.clone(), k_out=q)
    for bad in (dict(rot_dim=7), dict(rot_dim=16, sections=(3, 4)), dict(rot_dim=16, scaling="other"),
                dict(rot_dim=16, scaling="by_parts"), dict(rot_dim=2, scaling="base"), dict(rot_dim=16, factor=0.0)):
        with pytest.raises(ValueError):
            sb.rotary_frequencies(**bad)
