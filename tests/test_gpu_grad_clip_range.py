"""Clips whose factor is below the normal fp32 numbers, against the definition."""
from __future__ import annotations

import sys

import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module")
def sb():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import seam_blending_patch_amd as m
    return m


def clipped(sb, grads, max_norm, out_dtypes):
    """The norm and the clipped gradients, in place where out_dtypes is None."""
    if out_dtypes is None:
        outs = [g.clone() for g in grads]
        return sb.grad_norm_clip(outs, max_norm, eps=EPS), outs
    outs = [torch.full(g.shape, 7.0, dtype=t, device="cuda") for g, t in zip(grads, out_dtypes)]
    return sb.grad_norm_clip(grads, max_norm, eps=EPS, out=outs), outs


@pytest.mark.parametrize("max_norm", [1e-3, 1e-6, 1e-8])
@pytest.mark.parametrize("out", ["place", "same", "fp32"])
def test_factors_below_the_normal_numbers(sb, max_norm, out):
    """Norms of about 7e37: factors of 1e-41, 1e-44 and 1e-46, of which fp32 holds
    13, 3 and no bits, while every result is a normal number.  The definition's
    bound: the norm's, the factor's and the product's rounding."""
    gen = torch.Generator().manual_seed(3)
    grads = [(torch.randn(n, generator=gen) * 1e36).to(t).cuda() for n, t in ((5000, F32), (3, BF16), (801, BF16))]
    grads += [torch.randn(77, generator=gen).to(F16).cuda()]
    print(f"[clip] factor of {max_norm} to 7e37, {out}", file=sys.stderr, flush=True)
    norm, tol, want, tols = ref.clip([ref.f64(g) for g in grads], max_norm, EPS)
    types = {"place": None, "same": [g.dtype for g in grads], "fp32": [F32] * len(grads)}[out]
    got, outs = clipped(sb, grads, max_norm, types)
    assert abs(got.item() - norm) <= tol
    for o, w, t in zip(outs, want, tols):
        ref.assert_near(o, w, t, f"{max_norm} {out}")
    assert abs(ref.f64(outs[0])).max() > 0


def test_norms_past_fp32(sb):
    """The norm is 64-bit inside: where it is past fp32 it reads as infinite, and
    the gradients still come out scaled to the bound."""
    grads = [torch.full((2000,), 3e38, device="cuda"), torch.full((9,), -1.0, device="cuda")]
    host = [ref.f64(g) for g in grads]
    _, _, want, tols = ref.clip(host, 2.0, EPS)
    norm, outs = clipped(sb, grads, 2.0, None)
    assert torch.isposinf(norm)
    for o, w, t in zip(outs, want, tols):
        ref.assert_near(o, w, t, "past fp32")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_factors_below_the_normal_numbers_and_not_finite_gradients(sb, bad):
    """An infinite element makes the norm infinite and the factor 0, as before."""
    grads = [torch.full((300,), 1e36, device="cuda")]
    grads[0][7] = bad
    norm, outs = clipped(sb, grads, 1e-8, None)
    if bad != bad:
        assert torch.isnan(norm) and torch.isnan(outs[0]).all()
    else:
        assert torch.isposinf(norm) and torch.isnan(outs[0][7])
        outs[0][7] = 0
        assert not outs[0].any()


def test_tensors_that_share_memory_are_refused_and_stay(sb):
    bucket = torch.randn(100, generator=torch.Generator().manual_seed(1)).cuda()
    before, other = bucket.clone(), torch.zeros(60, device="cuda")
    grads = [bucket[:60], bucket[56:]]
    for call in (lambda: sb.grad_norm_clip(grads, 1e-3), lambda: sb.GradNormClip(grads, 1e-3)(),
                 lambda: sb.grad_norm_clip([other, bucket[:60]], 1e-3, out=[bucket[40:], other])):
        with pytest.raises(sb.SeamBlendError) as e:
            call()
        assert e.value.code == -1 and "shares memory" in str(e.value)
    assert torch.equal(bucket, before) and not other.any()
    # read alone, or written elsewhere, they may
    want = ref.clip([ref.f64(g) for g in grads], 1e-3, EPS)
    norm, outs = clipped(sb, grads, 1e-3, [F32, F32])
    assert abs(norm.item() - want[0]) <= want[1] and torch.equal(sb.grad_norm(grads), norm)
    for o, w, t in zip(outs, want[2], want[3]):
        ref.assert_near(o, w, t, "shared")
