"""attention where most of the keys have weights far below the largest one."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

KEYS, GAP = 30000, 17.5


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def sink(queries, d, at, dtype):
    """one key with a value of 0 and a weight of nearly 1, 29999 others of 2.5e-8 each with
    values of 1; and what these weigh in all, 7.5e-4.  Queries alike: every row says the
    same; few rows take splits, 140000 the blocks of eight waves."""
    q = torch.zeros(1, queries, 1, d, dtype=dtype)
    k, v = torch.zeros(1, KEYS, 1, d, dtype=dtype), torch.ones(1, KEYS, 1, d, dtype=dtype)
    q[..., 0], k[0, at, 0, 0], v[0, at] = 1.0, GAP, 0.0
    rest = (KEYS - 1) * torch.exp(torch.tensor(-GAP, dtype=torch.float64))
    return q.cuda(), k.cuda(), v.cuda(), rest.item()


PLACES = [(n, d, at) for n in (1, 40, 300) for d in (64, 128, 160, 256) for at in (0, 11111, 29999)] \
    + [(140000, d, 11111) for d in (64, 128, 160)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("queries,d,at", [p for p in PLACES if p[1] in (64, 128)], ids=str)
def test_the_log_sum(sb, queries, d, at, dtype):
    """a tile's weights (16 or 32 of a lane) are added up before they are added to the
    rest: at most KEYS / 32 + 32 roundings of the whole in fp32, and a few of the score's
    and the logarithm's"""
    q, k, v, rest = sink(queries, d, at, dtype)
    _, lse = sb.attention(q, k, v, scale=1.0, return_lse=True)
    want = GAP + torch.log1p(torch.tensor(rest, dtype=torch.float64)).item()
    assert (lse.double() - want).abs().max().item() <= (KEYS / 32 + 32) * 2.0 ** -24 + 8 * 2.0 ** -24 * GAP


@pytest.mark.parametrize("queries,d,at", PLACES, ids=str)
def test_many_fp16_keys_below_one(sb, queries, d, at):
    """their weights lie below half of the smallest fp16 number"""
    q, k, v, rest = sink(queries, d, at, torch.float16)
    out = sb.attention(q, k, v, scale=1.0)
    # each weight is held in steps of 2^-24 over 2^7, off by half a step (0.9% of it); the
    # rest is some roundings of fp32 and the result's own, half a step of 2^-21
    assert (out.double() - rest / (1 + rest)).abs().max().item() <= (KEYS - 1) * 2.0 ** -32 * (1 + 1e-3) + 2.0 ** -22


def test_the_largest_weights_stay_finite(sb):
    """scores that grow by just less than what moves the running maximum: P passes through
    its largest value, 2^15, and sums of it stay in fp32"""
    n, d = 4096, 64
    q, k = torch.zeros(1, 64, 1, d, dtype=torch.float16), torch.zeros(1, n, 1, d, dtype=torch.float16)
    q[..., 0] = 1.0
    k[0, :, 0, 0] = torch.arange(n) // 64 * 5.5  # a tile's keys alike, each tile 2^7.9 of the last
    v = torch.randn(1, n, 1, d, generator=torch.Generator().manual_seed(1)).half()
    out = sb.attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
    p = torch.softmax(k[0, :, 0, 0].double(), 0)
    want = p @ v[0, :, 0].double()
    size = p @ v[0, :, 0].double().abs()
    # a rounding of P, of the score (352 at most) in base 2, and of the result
    assert ((out.double().cpu()[0, :, 0] - want).abs() <= size * (2.0 ** -11 * 2 + 4 * 352 * 2.0 ** -23)).all()
