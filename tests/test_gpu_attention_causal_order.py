"""causal attention whose tiles are put side by side by length: every tile is done once,
whatever the order, with some tiles over and with none; and sizes beyond the rule."""
from __future__ import annotations

import pytest
import torch

import attention_ref as ref
from transformer_ref import assert_near

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


# 8 units on 256 CUs, 32 to a unit; tiles of 128 rows of 8 heads: tokens / 16 tiles
SIZES = [(512, 32), (528, 33), (640, 40), (1024, 64), (1030, 65), (1120, 70), (1280, 80), (1296, 81)]


@pytest.mark.parametrize("tokens,tiles", SIZES, ids=str)
@pytest.mark.parametrize("d,dtype", [(32, "fp32"), (80, "fp32"), (128, "fp32"), (160, "fp32"), (64, "bf16"), (256, "bf16")], ids=str)
def test_every_tile_once(sb, tokens, tiles, d, dtype):
    assert torch.cuda.get_device_properties(0).multi_processor_count == 256 and -(-tokens * 8 // 128) == tiles
    gen = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda").to(DT[dtype])  # noqa: E731
    q, k, v = n(1, tokens, 64, d), n(1, tokens, 8, d), n(1, tokens, 8, d)
    out, lse = (torch.full(s, float("nan"), device="cuda", dtype=t) for s, t in ((q.shape, DT[dtype]), ((1, 64, tokens), torch.float32)))
    sb.attention(q, k, v, causal=True, out=out, lse=lse)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for y in (0, 7):  # key heads that are compared
        heads, own = slice(8 * y, 8 * y + 2), slice(y, y + 1)
        (o, s), (to, ts) = ref.forward(q[:, :, heads].cpu(), k[:, :, own].cpu(), v[:, :, own].cpu(), d ** -0.5, True)
        assert_near(out[:, :, heads], o, to, f"{tokens} {d} {dtype} out")
        assert_near(lse[:, heads], s, ts, f"{tokens} {d} {dtype} lse")
