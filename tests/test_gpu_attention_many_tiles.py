"""attention and its gradient where blocks are full and go over many tiles: the steady
state of the pipelines, against the 64-bit definition for some of the heads."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_ref as ref
from transformer_ref import assert_near

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def units(hq, hk, b, nq, rows):
    """blocks of `rows` rows (queries times the heads that share a key head)"""
    return b * hk * -(-nq * (hq // hk) // rows)


def draw(seed, b, nq, nk, hq, hk, d, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    q, k, v, g = n(b, nq, hq, d), n(b, nk, hk, d), n(b, nk, hk, d) + 0.5 * n(b, 1, hk, d), n(b, nq, hq, d)
    return [t.to(DT[dtype]) for t in (q, k, v, g)]


def run(sb, size, dtype, causal, lengths=None, backward=True):
    b, nq, nk, hq, hk, d = size
    q, k, v, g = draw(31, *size, dtype)
    how = dict(causal=causal)
    ql = kl = None
    if lengths:
        ql, kl = lengths
        for x in range(b):
            q[x, ql[x]:] = g[x, ql[x]:] = float("nan")
            k[x, kl[x]:] = v[x, kl[x]:] = float("inf")
        how |= dict(query_lengths=torch.tensor(ql, dtype=torch.int32, device="cuda"),
                    key_lengths=torch.tensor(kl, dtype=torch.int32, device="cuda"))
    out, lse = sb.attention(q, k, v, return_lse=True, **how)
    grads = sb.attention_backward(g, q, k, v, out, lse, **how) if backward else None
    group, scale = hq // hk, d ** -0.5
    for x, y in {(0, 0), (b - 1, hk - 1), (b // 2, hk // 2)}:  # samples and key heads that are looked at
        heads = slice(y * group, (y + 1) * group)
        of = lambda t, h: torch.nan_to_num(t[x:x + 1, :, h].cpu(), 0.0, 0.0, 0.0)  # noqa: E731
        own = of(q, heads), of(k, slice(y, y + 1)), of(v, slice(y, y + 1))
        l2 = (None, None) if ql is None else (ql[x:x + 1], kl[x:x + 1])
        (o, s), (to, ts) = ref.forward(*own, scale, causal, *l2)
        what = f"{size} {dtype} sample {x} key head {y}"
        assert_near(lse[x:x + 1, heads], s, ts, what + " lse")
        assert_near(out[x:x + 1, :, heads], o, to, what + " out")
        if backward:
            # (the definition's bounds leave dout's products with the rounded out its rounding)
            want, tol = ref.backward(of(g, heads), *own, of(out, heads), lse[x:x + 1, heads].cpu(), scale, causal, *l2)
            parts = grads[0][x:x + 1, :, heads], grads[1][x:x + 1, :, y:y + 1], grads[2][x:x + 1, :, y:y + 1]
            for name, a, w, t in zip(("dq", "dk", "dv"), parts, want, tol):
                assert_near(a, w, t, f"{what} {name}")
    # the heads that were not looked at: finite, and zeros where lengths leave nothing
    assert torch.isfinite(out).all()
    if lengths:
        for x in range(b):
            assert not out[x, ql[x]:].any()
            if backward:
                assert not grads[0][x, ql[x]:].any() and not grads[1][x, kl[x]:].any() and not grads[2][x, kl[x]:].any()


@pytest.fixture(scope="module")
def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


# heads of 96 and 128 take tiles of 64 keys, longer ones of 32: five tiles at least, the
# last one cut; rows that fill both sets of a block's waves, and leave the last block short
WIDE = [(1, 4100, 333, 32, 32, 128), (1, 4100, 333, 32, 32, 96), (1, 4100, 397, 32, 32, 104), (1, 4100, 170, 32, 32, 160),
        (1, 4100, 233, 32, 32, 192), (4, 1100, 401, 32, 8, 128), (1, 4128, 640, 32, 32, 128)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", WIDE, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_blocks_of_eight_waves(sb, cus, dtype, size, causal):
    b, nq, nk, hq, hk, d = size
    assert units(hq, hk, b, nq, 256) >= 2 * cus and nk > 4 * (64 if d <= 128 else 32)
    run(sb, size, dtype, causal)


LONG = [
    # causal rows that see from one to all of 15 tiles; keys' gradients over 22 tiles of rows
    (8, 700, 900, 32, 32, 128), (8, 700, 900, 32, 32, 64), (8, 700, 500, 32, 32, 160), (8, 300, 900, 64, 32, 96),
]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", LONG, ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_long_rows_and_columns(sb, cus, dtype, size, causal):
    b, nq, nk, hq, hk, d = size
    assert units(hq, hk, b, nq, 256) >= 2 * cus  # (nothing is split)
    run(sb, size, dtype, causal)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("size", [(8, 700, 900, 32, 32, 128), (8, 700, 500, 32, 32, 160), (8, 700, 900, 32, 32, 64)], ids=str)
@pytest.mark.parametrize("causal", [False, True])
def test_lengths_that_end_in_later_tiles(sb, cus, dtype, size, causal):
    b, nq, nk, hq, hk, d = size
    assert units(hq, hk, b, nq, 256) >= 2 * cus
    ql = [min(n, nq) for n in (700, 1, 513, 0, 385, 256, 129, 699)]
    kl = [min(n, nk) for n in (450, 900, 1, 333, 0, 321, 899, 257)]
    run(sb, size, dtype, causal, (ql, kl))


def test_dq_of_short_heads(sb, cus):
    """heads of up to 64 over eleven tiles of keys"""
    size = (1, 4100, 333, 32, 32, 64)
    assert units(32, 32, 1, 4100, 256) >= 2 * cus
    for dtype in DT:
        for causal in (False, True):
            run(sb, size, dtype, causal)
            run(sb, (1, 4100, 333, 32, 32, 32), dtype, causal)


@pytest.mark.parametrize("dtype", DT)
def test_many_tiles_the_same_bits(sb, dtype):
    q, k, v, g = draw(5, 8, 700, 900, 32, 32, 128, dtype)
    out, lse = sb.attention(q, k, v, causal=True, return_lse=True)
    grads = sb.attention_backward(g, q, k, v, out, lse, causal=True)
    for _ in range(4):
        again = sb.attention(q, k, v, causal=True, return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
        for a, b in zip(sb.attention_backward(g, q, k, v, out, lse, causal=True), grads):
            assert torch.equal(a, b)
