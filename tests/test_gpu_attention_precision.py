"""attention_backward in 16 bits where the rounding of `out` would weigh most: values
and keys with a large mean.  dq and dk are as exact as their own roundings and those of
dS allow, whatever `out` was rounded to."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
from transformer_ref import U, assert_near, f64

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def backward(dout, q, k, v, out, scale, causal, q_len=None, k_len=None, tiny=None):
    """((dq, dk), tolerances); tiny: what P, dS of dq and dS of dk may lose below the
    normal numbers (arrays of [B, heads, Lq, 1]), by default fp16's.  With delta' the row sums of dout and the rounded out,
    dS' = P (dp - delta') is off by E = |delta - delta'| times P, which its own sum takes
    out again:
      dq = sum dS' k - r m, r = sum dS' (rounded), m = sum P k (P rounded);
      dk = sum P (dp - delta' - sum dS') q.
    So E itself is nowhere an error, but dS' and P are rounded (h of each), and r and m
    take those roundings along."""
    dt, h = q.dtype, ref.HALF[q.dtype]
    tinies = [np.full((q.shape[0], q.shape[2], q.shape[1], 1), ref.TINY[dt])] * 3 if tiny is None else tiny
    ql, kl = ref.lengths(q_len, k_len, q, k)
    group, d = q.shape[2] // k.shape[2], q.shape[3]
    dq, dk = np.zeros(q.shape), np.zeros(k.shape)
    tq, tk = np.zeros(q.shape), np.zeros(k.shape)
    q, k, v, g, out = (f64(t) for t in (q, k, v, dout, out))
    for b, (nq, nk) in enumerate(zip(ql, kl)):
        for x in range(q.shape[2] if nq and nk else 0):
            y = x // group
            tiny_p, tiny_q, tiny_k = (t[b, x, :nq] for t in tinies)
            qq, kk, vv, gg, oo = q[b, :nq, x], k[b, :nk, y], v[b, :nk, y], g[b, :nq, x], out[b, :nq, x]
            p, ls, off, seen = ref.probabilities(qq, kk, scale, causal, dt)
            off = off + 4 * U * np.abs(np.where(np.isfinite(ls), ls, 0.0))[:, None]
            dp = gg @ vv.T
            size = np.abs(gg) @ np.abs(vv).T  # what dp's terms sum up to
            delta, near = (p * dp).sum(1, keepdims=True), (gg * oo).sum(1, keepdims=True)
            e = np.abs(delta - near) + (d + 4) * U * (np.abs(gg) * np.abs(oo)).sum(1, keepdims=True)
            ds = p * (dp - delta)
            most = np.abs(ds) + p * e  # |dS'|
            own = (d + 8) * U * size + 4 * U * (np.abs(dp) + np.abs(near))  # of dp - delta', before the rounding
            err = off * most + p * own
            rounded = err + (h + 2 * U) * (most + err) + tiny_q * seen + (nk + 8) * U * most
            e_p = (off + h + (nk + 8) * U) * p + tiny_p * seen
            m = p @ np.abs(kk)
            dq[b, :nq, x] = scale * ds @ kk
            tq[b, :nq, x] = scale * (rounded @ np.abs(kk) + rounded.sum(1, keepdims=True) * (m + e_p @ np.abs(kk))
                                     + e * (e_p @ np.abs(kk)) + 4 * U * e * m)
            e_sum = (err + (nk + 8) * U * most).sum(1, keepdims=True) + 2 * U * np.abs(delta)
            err = off * np.abs(ds) + p * (own + e_sum)
            err = err + (h + 2 * U) * (np.abs(ds) + err) + tiny_k * seen
            rows = nq * group
            dk[b, :nk, y] += scale * ds.T @ qq
            tk[b, :nk, y] += scale * ((err + (rows + 8) * U * np.abs(ds)).T @ np.abs(qq))
    return (dq, dk), (tq, tk)


def draw(seed, b, nq, nk, hq, hk, d, dtype, mean):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    q, k, v, g = n(b, nq, hq, d), n(b, nk, hk, d) + 1.0, n(b, nk, hk, d) + mean, n(b, nq, hq, d)
    return [t.to(DT[dtype]) for t in (q, k, v, g)]


SIZES = [
    # b, queries, keys, heads, key heads, D: blocks for many rows, split, few rows, heads of
    # odd length, heads that take two waves; shared key heads
    (8, 300, 300, 32, 32, 64), (1, 200, 260, 4, 2, 64), (4, 260, 230, 16, 16, 128), (1, 300, 290, 2, 2, 96),
    (2, 200, 210, 2, 1, 160), (1, 190, 200, 2, 2, 192), (1, 150, 140, 2, 1, 33), (1, 140, 150, 1, 1, 127),
    (1, 150, 170, 2, 2, 161), (1, 170, 150, 2, 1, 256), (1, 1, 1500, 8, 2, 128), (1, 3, 900, 4, 4, 256),
    (1, 2, 700, 2, 1, 191), (1, 1200, 40, 2, 2, 64),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_a_large_mean_of_values_and_keys(sb, dtype, size, causal):
    q, k, v, g = draw(1, *size, dtype, 64.0)
    scale = size[-1] ** -0.5
    (out, lse), _ = ref.forward(q, k, v, scale, causal)
    out, lse = torch.from_numpy(out).to(q.dtype), torch.from_numpy(lse).float()
    want, tol = backward(g, q, k, v, out, scale, causal)
    got = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse)), causal=causal)
    for name, a, w, t in zip(("dq", "dk"), got, want, tol):
        assert_near(a, w, t, f"{size} {dtype} {name}")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(4, 300, 300, 8, 4, 64), (3, 1, 1500, 8, 2, 128), (3, 140, 150, 2, 2, 256)], ids=str)
def test_a_large_mean_and_unlike_lengths(sb, dtype, size):
    q, k, v, g = draw(2, *size, dtype, -30.0)
    ql, kl = [size[1], size[1] // 2, 0, 1][:size[0]], [size[2] // 3, size[2], 40, 3][:size[0]]
    scale = size[-1] ** -0.5
    (out, lse), _ = ref.forward(q, k, v, scale, True, ql, kl)
    out, lse = torch.from_numpy(out).to(q.dtype), torch.from_numpy(lse).float()
    want, tol = backward(g, q, k, v, out, scale, True, ql, kl)
    lens = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in (ql, kl)]
    got = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse)), causal=True, query_lengths=lens[0],
                                key_lengths=lens[1])
    for name, a, w, t in zip(("dq", "dk"), got, want, tol):
        assert_near(a, w, t, f"{size} {dtype} {name}")


@pytest.mark.parametrize("dtype", DT)
def test_one_key_has_no_gradient(sb, dtype):
    """its weight is 1 whatever the scores, and out is its value, which 16 bits hold: dS
    is what fp32 leaves of dout v - delta, and dq and dk a rounding of nothing"""
    q, k, v, g = draw(3, 2, 70, 1, 4, 2, 64, dtype, 64.0)
    out = v.repeat_interleave(2, 2).expand(q.shape).contiguous()
    lse = torch.einsum("bqhd,bkhd->bhqk", q.double(), k.repeat_interleave(2, 2).double())[..., 0] * 0.125
    dq, dk, dv = sb.attention_backward(*(t.cuda() for t in (g, q, k, v, out, lse.float())))
    size = (g.double().abs() * out.double().abs()).sum(-1).max()
    assert f64(dq).__abs__().max() <= 0.125 * 140 * U * size * float(k.abs().max())
    assert f64(dk).__abs__().max() <= 0.125 * 140 * U * size * float(q.double().abs().sum((1, 2)).max()) * 2
