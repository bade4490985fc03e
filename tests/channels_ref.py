"""Plain 64-bit definitions (numpy) of the channels-last group norm with its
gradient and of dropout, with the error bounds the tests allow the kernels.

U is fp32's unit roundoff.  Roundings that add up in a statistic: a thread's
batch of 8 positions (8 sums each pass), 3 operations for each of its batches (at
most 8 in these tests' sizes), 3 for each of the at most 8 levels of a block's
tree, and the few around: below 80.
"""
from __future__ import annotations

import numpy as np

from transformer_ref import U

CHAIN = 80


def logistic(z):
    return 0.5 * (1 + np.tanh(0.5 * z))


def statistics(x, groups, eps):
    """(h, 1 / sigma, error of h) of x [N, S, C], the latter two by element."""
    n, s, c = x.shape
    v = x.reshape(n, s, groups, c // groups)
    mean = v.mean((1, 3), keepdims=True)
    var = ((v - mean) ** 2).mean((1, 3), keepdims=True)
    r = 1 / np.sqrt(var + eps)
    h = (v - mean) * r
    # sums are of differences from the group's first value, `shift` sigmas from the mean
    shift = np.abs(v[:, :1, :, :1] - mean) * r
    err = CHAIN * U * (1 + np.abs(h) + shift)
    return h.reshape(x.shape), np.broadcast_to(r, v.shape).reshape(x.shape), err.reshape(x.shape)


def group_norm(x, groups, gamma, beta, eps, silu):
    """(y, tolerance)"""
    h, _, err = statistics(x, groups, eps)
    g, b = (1.0 if gamma is None else gamma), (0.0 if beta is None else beta)
    z = h * g + b
    tol = err * np.abs(g) + 4 * U * (np.abs(h * g) + np.abs(b))
    if not silu:
        return z, tol
    s = logistic(z)
    # |act'| <= 1.1; the logistic's argument is off by 2 |z| U, itself by 4 U
    return z * s, 1.1 * tol + np.abs(z) * (s * (1 - s) * (2 * np.abs(z) + 4) + 4 * s) * U + 1e-30


def group_norm_backward(dy, x, groups, gamma, beta, eps, silu):
    """((dx, dgamma, dbeta), tolerances)"""
    h, r, e_h = statistics(x, groups, eps)
    ga, b = (1.0 if gamma is None else gamma), (0.0 if beta is None else beta)
    g, e_g = dy, np.zeros_like(dy)
    if silu:
        z = h * ga + b
        e_z = e_h * np.abs(ga) + 4 * U * (np.abs(h * ga) + np.abs(b))
        s = logistic(z)
        # |act''| <= 0.5; act' = s (1 + z (1 - s)) with s as above
        g = dy * s * (1 + z * (1 - s))
        e_g = np.abs(dy) * (0.5 * e_z + 8 * U * (1 + np.abs(z)) * (s * (1 - s) * (1 + np.abs(z)) + s) + 4 * U)
    a, e_a = g * ga, e_g * np.abs(ga) + 2 * U * np.abs(g * ga)
    n, sz, c = x.shape
    over = lambda t: np.broadcast_to(t.reshape(n, sz, groups, c // groups).mean((1, 3), keepdims=True),  # noqa: E731
                                     (n, sz, groups, c // groups)).reshape(x.shape)
    ma, mah = over(a), over(a * h)
    e_ma = over(e_a + CHAIN * U * np.abs(a))
    e_mah = over(e_a * np.abs(h) + np.abs(a) * e_h + CHAIN * U * np.abs(a * h))
    inner = a - ma - h * mah
    size = np.abs(a) + np.abs(ma) + np.abs(h * mah)
    tol = r * (e_a + e_ma + np.abs(h) * e_mah + e_h * np.abs(mah) + 4 * U * size) + CHAIN * U * r * np.abs(inner)
    return ((r * inner, (g * h).sum((0, 1)), g.sum((0, 1))),
            (tol, (e_g * np.abs(h) + np.abs(g) * e_h + CHAIN * U * np.abs(g * h)).sum((0, 1)),
             (e_g + CHAIN * U * np.abs(g)).sum((0, 1))))


def philox(counter, key):
    """Philox4x32 with ten rounds: counters [n, 4] and a key of two 32-bit words
    -> words [n, 4]."""
    m = np.uint64(0xFFFFFFFF)
    a, b, c, d = (counter[:, k].astype(np.uint64) for k in range(4))
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        p, q = a * np.uint64(0xD2511F53), c * np.uint64(0xCD9E8D57)
        a, b, c, d = (q >> np.uint64(32)) ^ b ^ np.uint64(k0), q & m, (p >> np.uint64(32)) ^ d ^ np.uint64(k1), p & m
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack((a, b, c, d), 1)


def words(n, seed, offset, site):
    """the generator's word of each of n elements"""
    at = np.arange((n + 3) // 4, dtype=np.uint64)
    full = lambda v: np.full_like(at, v)  # noqa: E731
    counter = np.stack((at, full(site), full(offset & 0xFFFFFFFF), full(offset >> 32 & 0xFFFFFFFF)), 1)
    return philox(counter, (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF)).reshape(-1)[:n]


def dropout(x, p, seed, offset, site, residual=None):
    """(y, tolerance): the factor is off by U, the product (and the sum) rounded once more."""
    keep = (words(x.size, seed, offset, site) >= int(np.floor(p * 2.0 ** 32))).reshape(x.shape)
    y = np.where(keep, x / (1 - p), 0.0)
    tol = 2 * U * np.abs(y)
    if residual is not None:
        y = y + residual
        tol = tol + U * np.abs(y)
    return y, tol
