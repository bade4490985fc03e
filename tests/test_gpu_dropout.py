"""dropout and dropout_backward against the generator's definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import channels_ref as ref
from transformer_ref import assert_near, f64

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SEED, OFFSET = 0x0123456789ABCDEF, 0x7EDCBA9876543210


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def state(seed=SEED, offset=OFFSET):
    return torch.tensor([seed, offset], device="cuda")


def draw(seed, shape, dtype):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(shape, generator=gen).to(DT[dtype]).cuda() for _ in range(2)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", [(1,), (3,), (7, 5), (77, 768), (1, 4099), (3, 2, 1023), (513, 16)], ids=str)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_against_the_definition(sb, dtype, shape, p):
    x, res = draw(1, shape, dtype)
    for residual in (None, res):
        want, tol = ref.dropout(f64(x), p, SEED, OFFSET, 5, None if residual is None else f64(residual))
        assert_near(sb.dropout(x, p, state(), site=5, residual=residual), want, tol, f"{shape} {p}")
    assert torch.equal(sb.dropout_backward(x, p, state(), site=5), sb.dropout(x, p, state(), site=5))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [1, 2, 3, 5, 8, 63, 64, 130])
def test_strided_rows_have_the_mask_of_dense_ones(sb, dtype, width):
    """also rows whose first element is in the middle of a counter's four words"""
    whole, res = draw(2, (5, 6, width + 3), dtype)
    x, r = whole[:, 1:5, 2:width + 2], res[:, :4, :width]
    want = sb.dropout(x.contiguous(), 0.3, state(), residual=r.contiguous())
    assert torch.equal(sb.dropout(x, 0.3, state(), residual=r), want)
    keep = whole.clone()
    assert sb.dropout(x, 0.3, state(), residual=r, out=x) is x
    assert torch.equal(x, want)
    keep[:, 1:5, 2:width + 2] = want
    assert torch.equal(whole, keep)
    assert sb.dropout(want, 0.3, state(), out=want) is want


def test_seeds_offsets_and_sites_differ(sb):
    x = torch.ones(4096, device="cuda")
    masks = [sb.dropout(x, 0.5, state(s, o), site=i) != 0 for s, o, i in
             ((1, 2, 0), (2, 2, 0), (1 + (1 << 32), 2, 0), (1, 3, 0), (1, 2 + (1 << 32), 0), (1, 2, 1), (-1, -1, 2 ** 32 - 1))]
    for a in range(len(masks)):
        # 4096 fair coins: 4096 / 2 agree, give or take 6 times their deviation of 32
        for b in range(a):
            assert abs(int((masks[a] == masks[b]).sum()) - 2048) <= 6 * 32
        assert abs(int(masks[a].sum()) - 2048) <= 6 * 32
    assert torch.equal(masks[0], sb.dropout(x, 0.5, state(1, 2)) != 0)
    neg = ref.words(16, -1 & (2 ** 64 - 1), -1 & (2 ** 64 - 1), 2 ** 32 - 1) >= 2 ** 31
    assert np.array_equal(masks[-1][:16].cpu().numpy(), neg)


def test_dropped_places_may_hold_anything(sb):
    x = torch.full((4096,), float("nan"), device="cuda")
    dropped = torch.from_numpy(ref.words(4096, SEED, OFFSET, 0) < 2 ** 31).cuda()
    y = sb.dropout(x, 0.5, state(), residual=torch.ones_like(x))
    assert (y[dropped] == 1).all() and torch.isnan(y[~dropped]).all()


def test_large(sb):
    """more than one grid of the smallest kind, past the caches; counters past 2^24"""
    n = (1 << 27) + 5
    x = torch.ones(n, dtype=torch.float16, device="cuda")
    y = sb.dropout(x, 0.25, state())
    tail = (1 << 27) - 3
    keep = ref.philox(np.stack([np.arange(tail // 4, n // 4 + 1, dtype=np.uint64)] + [np.full(n // 4 + 1 - tail // 4, v, np.uint64)
                                for v in (0, OFFSET & 0xFFFFFFFF, OFFSET >> 32)], 1),
                      (SEED & 0xFFFFFFFF, SEED >> 32)).reshape(-1)[tail % 4:][:n - tail] >= 2 ** 30
    assert np.array_equal((y[tail:] != 0).cpu().numpy(), keep)
    share = float((y == 0).float().mean())
    assert abs(share - 0.25) <= 6 * (0.25 * 0.75 / n) ** 0.5 + 2.0 ** -24  # (the mean of 2^27 in fp32)


def test_a_captured_call_moves_with_its_offset(sb):
    x, res = draw(3, (33, 65), "bf16")
    st = state(9, 0)
    call = sb.Dropout(x, 0.2, st, site=3, residual=res)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st[1].add_(1)
        call()
    seen = []
    for turn in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(call.out, sb.dropout(x, 0.2, state(9, turn + 1), site=3, residual=res))
        seen.append(call.out.clone())
    assert not any(torch.equal(a, b) for a, b in zip(seen, seen[1:]))


def test_writes_raise_the_version(sb):
    x, y = draw(4, (8, 8), "fp32")
    st = state()
    for call in (lambda: sb.dropout(x, 0.5, st, out=y), lambda: sb.dropout_backward(x, 0.5, st, dx=y),
                 sb.Dropout(x, 0.5, st, out=y)):
        before, read = y._version, (x._version, st._version)
        call()
        assert y._version > before and (x._version, st._version) == read


def test_refusals(sb):
    x, y = draw(5, (8, 8), "fp32")
    st = state()
    bad = [
        (TypeError, lambda: sb.dropout(x.cpu(), 0.5, st)), (TypeError, lambda: sb.dropout(x.double(), 0.5, st)),
        (ValueError, lambda: sb.dropout(x[0, 0], 0.5, st)), (ValueError, lambda: sb.dropout(x, 0.5, st.int())),
        (ValueError, lambda: sb.dropout(x, 0.5, st.cpu())), (ValueError, lambda: sb.dropout(x, 0.5, st[:1])),
        (ValueError, lambda: sb.dropout(x, 0.5, st, site=-1)), (ValueError, lambda: sb.dropout(x, 0.5, st, site=1 << 32)),
        (ValueError, lambda: sb.dropout(x, 0.5, st, residual=y.half())), (ValueError, lambda: sb.dropout(x, 0.5, st, out=y[:4])),
        (ValueError, lambda: sb.dropout(x.t()[::2], 0.5, st)),
        (sb.SeamBlendError, lambda: sb.dropout(x, 1.0, st)), (sb.SeamBlendError, lambda: sb.dropout(x, -0.1, st)),
        (sb.SeamBlendError, lambda: sb.dropout(x, float("nan"), st)),
        (sb.SeamBlendError, lambda: sb.dropout(x[1:], 0.5, st, out=x[:-1])),
        (sb.SeamBlendError, lambda: sb.dropout(x[1:], 0.5, st, residual=y[1:], out=y[:-1])),
        (sb.SeamBlendError, lambda: sb.dropout(x, 0.5, st, out=y[:1].expand(8, 8))),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k} was not refused")
    assert sb.dropout(x[:0], 0.5, st).shape == (0, 8)
