"""Plain 64-bit definition of attention and its gradient, sample by sample and
head by head, with the error bounds the tests allow the kernels, term by term.

U is fp32's unit roundoff, H half a step of the storage type relative to a value
(nothing for fp32, whose operands are not rounded on the way).  A sum of n
terms, however it is ordered, is off by at most n U of its terms' magnitudes.
"""
from __future__ import annotations

import numpy as np
import torch

from transformer_ref import U, f64

# eps / 2: bf16 keeps 8 significant bits, so 1 and the next number are 2^-7 apart
# and a value just above 1 is rounded by up to 2^-8 of itself; fp16 keeps 11.
HALF = {torch.float32: 0.0, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
#: what a probability (or its gradient) of fp16 may lose below the normal numbers
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}


def lengths(q_len, k_len, q, k):
    b = q.shape[0]
    ql = [q.shape[1]] * b if q_len is None else [min(max(int(n), 0), q.shape[1]) for n in q_len]
    kl = [k.shape[1]] * b if k_len is None else [min(max(int(n), 0), k.shape[1]) for n in k_len]
    return ql, kl


def probabilities(q, k, scale, causal, dtype):
    """(P, log sums, relative error of P, seen) of one head's [queries, D], [keys, D]."""
    nq, nk, d = len(q), len(k), q.shape[1]
    s = scale * (q @ k.T)
    seen = np.ones((nq, nk), bool) if not causal else np.arange(nk) <= np.arange(nq)[:, None] + (nk - nq)
    s = np.where(seen, s, -np.inf)
    most = s.max(1, initial=-np.inf)
    base = np.where(np.isfinite(most), most, 0.0)
    e = np.exp(s - base[:, None])
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = base + np.log(total)
    p = e / np.where(total == 0, 1.0, total)[:, None]
    # a score: a sum of D products; its exponent in base 2 and the maximum's (or the
    # log sum's): a rounding each of a few operations, of their own size
    size = scale * (np.abs(q) @ np.abs(k).T)
    off = (d + 4) * U * size + 8 * U * (np.abs(np.where(seen, s, 0.0)) + np.abs(base)[:, None]) + 8 * U
    return p, np.where(total == 0, -np.inf, lse), np.where(seen, off, 0.0).max(1, initial=0.0)[:, None], seen


def forward(q, k, v, scale, causal=False, q_len=None, k_len=None):
    """((out, lse), tolerances) of torch tensors [B, T, heads, D]."""
    dt, h = q.dtype, HALF[q.dtype]
    ql, kl = lengths(q_len, k_len, q, k)
    group = q.shape[2] // k.shape[2]
    out = np.zeros(q.shape)
    lse = np.full((q.shape[0], q.shape[2], q.shape[1]), -np.inf)
    tol, tol_lse = np.zeros(out.shape), np.zeros(lse.shape)
    q, k, v = f64(q), f64(k), f64(v)
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        for x in range(q.shape[2] if nq and nk else 0):
            qq, kk, vv = q[b, :nq, x], k[b, :nk, x // group], v[b, :nk, x // group]
            p, ls, off, seen = probabilities(qq, kk, scale, causal, dt)
            out[b, :nq, x], lse[b, x, :nq] = p @ vv, ls
            pv = p @ np.abs(vv)
            # P and the sum that divides it are off by `off` each, both sums by nk U;
            # the largest P is 1 at least when fp16 loses its small ones
            tol[b, :nq, x] = (2 * off + h + (2 * nk + 8) * U) * pv + TINY[dt] * (seen @ np.abs(vv))
            tol_lse[b, x, :nq] = np.where(np.isfinite(ls), off[:, 0] + (nk + 8) * U
                                          + 4 * U * np.abs(np.where(np.isfinite(ls), ls, 0)), 0.0)
    return (out, lse), (tol, tol_lse)


def backward(dout, q, k, v, out, lse, scale, causal=False, q_len=None, k_len=None):
    """((dq, dk, dv), tolerances).  ``out`` and ``lse`` are what the kernel is given:
    out is off by half a step, lse by a rounding."""
    dt, h, tiny = q.dtype, HALF[q.dtype], TINY[q.dtype]
    ql, kl = lengths(q_len, k_len, q, k)
    group, d = q.shape[2] // k.shape[2], q.shape[3]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    tq, tk, tv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    q, k, v, g, out, lse = f64(q), f64(k), f64(v), f64(dout), f64(out), f64(lse)
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        for x in range(q.shape[2] if nq and nk else 0):
            y = x // group
            qq, kk, vv, gg = q[b, :nq, x], k[b, :nk, y], v[b, :nk, y], g[b, :nq, x]
            p, ls, off, seen = probabilities(qq, kk, scale, causal, dt)
            off = off + 4 * U * np.abs(np.where(np.isfinite(ls), ls, 0.0))[:, None]
            dp = gg @ vv.T
            delta = (p * dp).sum(1, keepdims=True)
            ds = p * (dp - delta)
            e_dp = (d + 4) * U * (np.abs(gg) @ np.abs(vv).T)
            e_delta = (np.abs(gg) * np.abs(out[b, :nq, x])).sum(1, keepdims=True) * (2 * HALF[dt] + (d + 4) * U) \
                + 2 * U * np.abs(delta)
            if dt == torch.float32:
                e_delta += 4 * U * (np.abs(gg) * np.abs(out[b, :nq, x])).sum(1, keepdims=True)
            err = p * (off * np.abs(dp - delta) + e_dp + e_delta + 4 * U * (np.abs(dp) + np.abs(delta)))
            err = err + (h + 2 * U) * (np.abs(ds) + err) + tiny * seen
            rows = nq * group
            dq[b, :nq, x] = scale * ds @ kk
            tq[b, :nq, x] = scale * ((err + (nk + 8) * U * np.abs(ds)) @ np.abs(kk))
            dk[b, :nk, y] += scale * ds.T @ qq
            tk[b, :nk, y] += scale * ((err + (rows + 8) * U * np.abs(ds)).T @ np.abs(qq))
            dv[b, :nk, y] += p.T @ gg
            tv[b, :nk, y] += ((off + h + (rows + 8) * U) * p + tiny * seen).T @ np.abs(gg)
    return (dq, dk, dv), (tq, tk, tv)
