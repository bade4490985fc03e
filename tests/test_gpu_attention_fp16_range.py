"""attention_backward in fp16 at the ends of its range: gradients and probabilities
far below its normal numbers, gradients whose products with the values pass 65504."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
from test_gpu_attention_precision import backward
from transformer_ref import U, assert_near, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def draw(seed, b, nq, nk, hq, hk, d, q=1.0, k=1.0, v=1.0, g=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda by, *s: (torch.randn(s, generator=gen) * by).half()  # noqa: E731
    return n(q, b, nq, hq, d), n(k, b, nk, hk, d), n(v, b, nk, hk, d), n(g, b, nq, hq, d)


def lifts(g, out, group):
    """What is lost below fp16's normal numbers, at most 2^-25: of P, which is held times
    2^14, and of dS, held times 2^4 over its row's norm of dout (dk: the largest row's),
    rounded up to a power of two, less where out's norm passes 2^8."""
    size = np.linalg.norm(f64(g), axis=-1) * np.maximum(1.0, np.linalg.norm(f64(out), axis=-1) / 256)
    size = np.maximum(size, 2.0 ** -30).transpose(0, 2, 1)
    most = size.reshape(size.shape[0], -1, group * size.shape[2]).max(2).repeat(group, 1)[:, :, None]
    step = lambda s: 2.0 ** -25 * 2.0 * s / 16.0  # noqa: E731
    return [np.full(size.shape + (1,), 2.0 ** -39), step(size)[..., None],
            np.broadcast_to(step(most)[..., None], size.shape + (1,))]


def check(sb, q, k, v, g, what, scale, causal=False):
    (out, lse), _ = ref.forward(q, k, v, scale, causal)
    out, lse = torch.from_numpy(out).half(), torch.from_numpy(lse).float()
    assert torch.isfinite(out).all()
    (dq, dk), (tq, tk) = backward(g, q, k, v, out, scale, causal, tiny=lifts(g, out, q.shape[2] // k.shape[2]))
    got = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse)), causal=causal, scale=scale)
    for name, a, w, t in zip(("dq", "dk"), got, (dq, dk), (tq, tk)):
        if np.abs(w).max() < 65000:
            assert_near(a, w, t, f"{what} {name}")
    return got


SIZES = [
    # b, queries, keys, heads, key heads, D
    (1, 64, 2048, 2, 1, 128), (4, 300, 300, 32, 32, 64), (1, 130, 540, 2, 1, 161), (1, 100, 700, 2, 2, 256),
    (1, 1, 3000, 4, 1, 64), (2, 2, 900, 2, 1, 33), (1, 900, 60, 2, 2, 40),
]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("which", ["dq", "dk"])
def test_small_gradients(sb, size, causal, which):
    """dout around 1e-5: dS lies below the smallest number of fp16, its products with
    large keys (queries) do not"""
    large, small = (30.0, 1 / 30.0) if which == "dq" else (1 / 30.0, 30.0)
    check(sb, *draw(1, *size, q=small, k=large, g=1e-5), f"{size}", size[-1] ** -0.5, causal)


@pytest.mark.parametrize("size", [(1, 10, 2, 2, 1, 64), (1, 70, 2, 1, 1, 128), (1, 10, 2, 2, 1, 161), (1, 8, 2, 1, 1, 256),
                                  (16, 300, 2, 32, 32, 64)], ids=str)
def test_large_gradients(sb, size):
    """dout around 1e4 (a scaled loss): dS passes 65504, the gradients do not"""
    got = check(sb, *draw(2, *size, q=0.01, k=0.01, v=8.0, g=1e4), f"{size}", size[-1] ** -0.5)
    assert all(torch.isfinite(t).all() for t in got[:2])


@pytest.mark.parametrize("size", [(1, 200, 700, 2, 1, 64), (1, 130, 140, 1, 1, 161), (1, 96, 600, 2, 2, 128)], ids=str)
def test_rows_of_unlike_gradients(sb, size):
    """rows of 1e-5 beside rows of 10 and of zeros"""
    q, k, v, g = draw(3, *size, q=1 / 30.0, k=30.0)
    by = torch.tensor([1e-5, 10.0, 0.0, 1e-3])[torch.arange(size[1]) % 4]
    check(sb, q, k, v, (g.float() * by[:, None, None]).half(), f"{size}", size[-1] ** -0.5)


@pytest.mark.parametrize("size", [(1, 70, 90, 2, 2, 128), (1, 40, 300, 1, 1, 256), (1, 33, 50, 1, 1, 64)], ids=str)
@pytest.mark.parametrize("g", [1e-3, 1.0])
def test_large_values(sb, size, g):
    """values with a mean of 600: norms of out of 5000 and more, and dS of ordinary size"""
    q, k, v, dout = draw(4, *size, g=g)
    got = check(sb, q, k, (v + 600.0), dout, f"{size}", size[-1] ** -0.5)
    assert all(torch.isfinite(t).all() for t in got)


@pytest.mark.parametrize("d", [64, 127, 256])
def test_small_probabilities(sb, d):
    """60000 keys of much the same weight, 1.7e-5 each: their values' gradients are P dout,
    a rounding of P and one of the result"""
    q, k, v, g = draw(5, 1, 1, 60000, 1, 1, d, q=0.2, g=30.0)
    (out, lse), _ = ref.forward(q, k, v, d ** -0.5)
    out, lse = torch.from_numpy(out).half(), torch.from_numpy(lse).float()
    p, ls, off, _ = ref.probabilities(f64(q)[0, :, 0], f64(k)[0, :, 0], d ** -0.5, False, torch.float16)
    want = p.T @ f64(g)[0, :, 0]
    tol = ((off + 4 * U * np.abs(ls)[:, None] + 2.0 ** -11 + 8 * U) * p + 2.0 ** -39).T @ np.abs(f64(g)[0, :, 0])
    dv = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse)))[2]
    assert_near(dv[0, :, 0], want, tol, "dv")


@pytest.mark.parametrize("d", [64, 161, 256])
def test_a_row_of_infinities_and_large_ones(sb, d):
    """causal order: keys behind an infinite row's last one have the gradients of the other
    rows, whose dS passes 65504"""
    q, k, v, g = draw(6, 1, 60, 60, 1, 1, d, q=0.01, k=0.01, v=8.0, g=2e3)
    g[0, 3] = float("inf")
    (out, lse), _ = ref.forward(q, k, v, d ** -0.5, True)
    out, lse = torch.from_numpy(out).half(), torch.from_numpy(lse).float()
    got = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse)), causal=True)
    clean = g.clone()
    clean[0, 3] = 0.0
    (dq, dk), (tq, tk) = backward(clean, q, k, v, out, d ** -0.5, True, tiny=lifts(clean, out, 1))
    rows = [i for i in range(60) if i != 3]
    assert not torch.isfinite(got[0][0, 3]).any() and not torch.isfinite(got[1][0, :4]).all()
    assert_near(got[0][:, rows], dq[:, rows], tq[:, rows], "dq")
    assert_near(got[1][:, 4:], dk[:, 4:], tk[:, 4:], "dk")


@pytest.mark.parametrize("size", [(3, 2, 1500, 4, 2, 64), (1, 200, 150, 4, 2, 128), (1, 900, 30, 2, 2, 33)], ids=str)
def test_a_captured_gradient_follows_the_scale(sb, size):
    """the powers of two are formed when the kernels run: a graph replayed on gradients of
    another scale gives what a call does"""
    scale = size[-1] ** -0.5
    q, k, v, g = (t.cuda() for t in draw(7, *size))
    out, lse = sb.attention(q, k, v, return_lse=True)
    back = sb.AttentionBackward(g, q, k, v, out, lse)
    back()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        back()
    for turn, by in enumerate((1.0, 1e-5, 1e3, 1e-2)):
        g.copy_(draw(8 + turn, *size, g=by)[3])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(back.out, sb.attention_backward(g, q, k, v, out, lse, scale=scale)):
            assert torch.equal(a, b)
