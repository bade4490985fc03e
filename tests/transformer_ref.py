"""Plain 64-bit definitions (numpy) of the transformer operators, with the
error bounds the tests allow the kernels, term by term.

U is fp32's unit roundoff.  A sum of n terms added in any order is off by at
most (n - 1) U times the sum of their magnitudes; the kernels' longest chains
are shorter (a lane's share, then trees), so the counts below are upper bounds.
"""
from __future__ import annotations

import numpy as np
import torch

import compare

U = 2.0 ** -24
NAME = {torch.float32: "fp32", torch.float16: "fp16", torch.bfloat16: "bf16"}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rounding(ref: np.ndarray, dtype: torch.dtype) -> np.ndarray:
    """Half a step of the storage type where the result may fall into the next
    binade (nothing for fp32, whose last rounding the bounds count)."""
    return np.zeros_like(ref) if dtype == torch.float32 else 0.5 * compare.ulp(np.abs(ref) * (1 + 2.0 ** -9), NAME[dtype])


def assert_near(got: torch.Tensor, ref: np.ndarray, tol: np.ndarray, what: str):
    assert tuple(got.shape) == ref.shape, f"{what}: shape {tuple(got.shape)}, expected {ref.shape}"
    g = f64(got)
    tol = tol + rounding(np.abs(ref) + tol, got.dtype)
    both = np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), both), f"{what}: finite in other places"
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{what}: NaN in other places"
    off = np.abs(g[both] - ref[both]) - tol[both]
    if off.size and off.max() > 0:
        k = int(np.argmax(off))
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {g.size} out of tolerance, worst: got "
                             f"{g[both].flat[k]!r}, expected {ref[both].flat[k]!r}, allowed {tol[both].flat[k]:.3g}")


def chain(d: int) -> int:
    """Roundings that add up in a row statistic: a lane's share of the row (at
    least 64 lanes from 512 elements on), the tree over lanes and waves, and the
    operations around."""
    return -(-d // 64) + 8 + 16


def layer_norm(x, gamma, beta, eps):
    """(y, tolerance): mean and variance are off by chain U of their size, so h
    by chain U (1 + |h|)."""
    d = x.shape[-1]
    m = x.mean(-1, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    h = (x - m) * r
    g = 1.0 if gamma is None else gamma
    y = h * g + (0.0 if beta is None else beta)
    return y, chain(d) * U * ((1 + np.abs(h)) * np.abs(g) + np.abs(y))


def layer_norm_backward(dy, x, gamma, eps):
    """((dx, dgamma, dbeta), tolerances).  Every mean over the row is off by
    chain U of the mean of its terms' magnitudes, a term with h by U (1 + |h|)
    chain more; a sum over n rows adds n U."""
    d, rows = x.shape[-1], x.size // x.shape[-1]
    m = x.mean(-1, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    h = (x - m) * r
    g = dy if gamma is None else dy * gamma
    mg, mgh = g.mean(-1, keepdims=True), (g * h).mean(-1, keepdims=True)
    dx = r * (g - mg - h * mgh)
    ah, ag = 1 + np.abs(h), np.abs(g)
    c = chain(d) * U
    tol_dx = 2 * c * r * (ag + ag.mean(-1, keepdims=True) + ah * (ag * ah).mean(-1, keepdims=True))
    over = tuple(range(x.ndim - 1))
    return ((dx, (dy * h).sum(over), dy.sum(over)),
            (tol_dx, (c + rows * U) * (np.abs(dy) * ah).sum(over), (rows + 8) * U * np.abs(dy).sum(over)))


def rotary(x, positions, freqs, sections, interleaved, scale, transpose=False):
    """(turned, tolerance) of [B, T, H, D] heads by [axes, B, T] positions.  The
    angle's last rounding is pi U, cosine and sine are good to 2 ulp, the scale,
    products and their sum add 4 roundings; before it the angle is rounded to 64
    bits a few times on either side (2^-50 of it in all)."""
    pairs = len(freqs)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.moveaxis(positions.astype(np.float64), 0, -1)[..., axis] * freqs
    c, s = np.cos(angle)[:, :, None] * scale, np.sin(angle)[:, :, None] * scale * (-1 if transpose else 1)
    first = slice(0, 2 * pairs, 2) if interleaved else slice(0, pairs)
    second = slice(1, 2 * pairs, 2) if interleaved else slice(pairs, 2 * pairs)
    u, v = x[..., first], x[..., second]
    out, tol = x.copy(), np.zeros_like(x)
    out[..., first], out[..., second] = u * c - v * s, u * s + v * c
    tol[..., first] = tol[..., second] = ((12 * U + 2.0 ** -50 * np.abs(angle))[:, :, None]
                                          * abs(scale) * (np.abs(u) + np.abs(v)))
    return out, tol


def clip(grads, max_norm, eps):
    """(norm, tolerance, scaled, tolerances): the sum is 64-bit, the norm and the
    factor are rounded once each, and every product once (to a step of 2^-149
    where it is that small)."""
    norm = np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
    by = min(1.0, max_norm / (norm + eps)) if np.isfinite(norm) else max_norm / (norm + eps)
    return norm, 2 * U * norm, [g * by for g in grads], [4 * U * np.abs(g * by) + 2.0 ** -149 for g in grads]
