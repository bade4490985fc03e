"""Attention, group norm and dropout at sizes whose offsets pass 32 bits or that take
more than one launch."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("queries", [1, 300])
def test_a_cache_past_32_bits(sb, queries):
    """one head of a cache of 256: its last keys begin 2.3 G elements from its first,
    bit for bit as from a dense copy, forward and backward"""
    keys, wide = 70000, 256 * 128
    assert keys * wide > 2 ** 31
    cache = torch.empty(2, keys, 256, 128, dtype=torch.bfloat16, device="cuda")
    k, v = (normal(s, 1, keys, 1, 128) for s in (1, 2))
    for at, t in zip(cache, (k, v)):
        at[:, 3:4] = t[0]
    fk, fv = (c[None, :, 3:4] for c in cache)
    q, g = normal(3, 1, queries, 4, 128), normal(4, 1, queries, 4, 128)
    want = sb.attention(q, k, v, causal=True, return_lse=True)
    got = sb.attention(q, fk, fv, causal=True, return_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ends = torch.tensor([keys - 5], dtype=torch.int32, device="cuda")
    assert torch.equal(sb.attention(q, fk, fv, key_lengths=ends), sb.attention(q, k[:, :-5], v[:, :-5]))
    dk, dv = (c[None, :, 9:10] for c in cache)  # the gradients into another head of it
    dq, _, _ = sb.attention_backward(g, q, fk, fv, *got, causal=True, dk=dk, dv=dv)
    for a, b in zip((dq, dk, dv), sb.attention_backward(g, q, k, v, *want, causal=True)):
        assert torch.equal(a, b)


def test_more_units_than_a_launch_takes(sb):
    """2^24 + 5 samples of one key: their results are the values"""
    n = (1 << 24) + 5
    q, k, v = (torch.randn(n, 1, 1, 2, device="cuda", dtype=torch.float16) for _ in range(3))
    out, lse = sb.attention(q, k, v, return_lse=True)
    assert torch.equal(out, v)
    score = (q.float() * k.float()).sum(-1).view(-1) * 0.5 ** 0.5
    # a sum of two products, its scaling and a few operations of the log sum
    assert (lse.view(-1) - score).abs().max() <= 8 * 2.0 ** -24 * (q.float() * k.float()).abs().sum(-1).max()
    _, _, dv = sb.attention_backward(q, q, k, v, out, lse)
    assert torch.equal(dv, q)  # (exp of a rounding is 1 in 16 bits)


def test_group_norm_past_32_bits(sb):
    """positions 2^15 elements apart: the last begin past 2^31, as from a dense copy"""
    whole = torch.empty(1, 70000, 1 << 15, dtype=torch.bfloat16, device="cuda")
    x, dy = normal(5, 1, 70000, 64), normal(6, 1, 70000, 64)
    far = whole[..., 100:164]
    far.copy_(x)
    y, stats = sb.group_norm(x, 8, activation="silu", return_stats=True)
    got, far_stats = sb.group_norm(far, 8, activation="silu", return_stats=True)
    assert torch.equal(got, y) and torch.equal(stats, far_stats)
    dx, dgamma, dbeta = sb.group_norm_backward(dy, x, 8, stats, activation="silu", weight_grads=True)
    into = whole[..., 300:364]
    got = sb.group_norm_backward(dy, far, 8, stats, activation="silu", weight_grads=True, dx=into)
    assert torch.equal(into, dx) and torch.equal(got[1], dgamma) and torch.equal(got[2], dbeta)


def test_many_samples(sb):
    """the most samples times groups that a call takes, a block to each"""
    n = (1 << 22) - (1 << 12)
    x = torch.randn(n, 4, 8, device="cuda", dtype=torch.float32)
    y, stats = sb.group_norm(x, 1, return_stats=True)
    want = torch.nn.functional.layer_norm(x.view(n, 32), (32,), eps=1e-6).view(n, 4, 8)
    assert (y - want).abs().max() <= 1e-5  # 32 values: some 20 roundings of numbers up to 6 on either side
    _, dgamma, dbeta = sb.group_norm_backward(torch.ones_like(x), x, 1, stats, weight_grads=True)
    assert torch.equal(dbeta, torch.full((8,), 4.0 * n, device="cuda"))
    with pytest.raises(sb.SeamBlendError):
        sb.group_norm(torch.empty(n + 1, 1, 8, device="cuda"), 1)


def test_dropout_rows_past_32_bits(sb):
    whole = torch.empty(70000, 1 << 15, dtype=torch.bfloat16, device="cuda")
    x = normal(7, 70000, 64)
    far = whole[:, 50:114]
    far.copy_(x)
    state = torch.tensor([3, 4], device="cuda")
    assert torch.equal(sb.dropout(far, 0.4, state), sb.dropout(x, 0.4, state))
