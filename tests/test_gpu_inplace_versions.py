"""What the transformer operators overwrite counts as written for torch's
autograd: a backward pass that saved it is refused, not computed from it."""
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


def heads(seed):
    return torch.randn(5, 3, 16, generator=torch.Generator().manual_seed(seed)).cuda()


def calls(sb):
    """(what a call overwrites, the call) for every way of giving a tensor to be written."""
    x, y, z, q, k = (heads(s) for s in range(5))
    row, bias = torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    f, _ = sb.rotary_frequencies(16)
    p = torch.arange(5, device="cuda")
    yield "layer_norm out", [y], lambda: sb.layer_norm(x, out=y)
    yield "layer_norm in place", [y], lambda: sb.layer_norm(y, out=y)
    yield "LayerNorm", [y], sb.LayerNorm(x, out=y)
    yield "layer_norm_backward dx", [z], lambda: sb.layer_norm_backward(y, x, dx=z)
    yield "layer_norm_backward all", [z, row, bias], lambda: sb.layer_norm_backward(y, x, dx=z, dgamma=row, dbeta=bias)
    yield "layer_norm_backward weights", [row, bias], lambda: sb.layer_norm_backward(y, x, dgamma=row, dbeta=bias)
    yield "LayerNormBackward", [z, row, bias], sb.LayerNormBackward(y, x, dx=z, dgamma=row, dbeta=bias)
    yield "rotary out", [y], lambda: sb.rotary(q, p, f, out=y)
    yield "rotary in place", [q, k], lambda: sb.rotary(q, p, f, k=k, out=q, k_out=k)
    yield "rotary key alone", [k], lambda: sb.rotary(q, p, f, k=k, k_out=k)
    yield "rotary_backward", [q, k], lambda: sb.rotary_backward(q, p, f, k=k, out=q, k_out=k)
    yield "Rotary", [q, k], sb.Rotary(q, p, f, k=k, out=q, k_out=k)
    yield "grad_norm_clip in place", [x, row], lambda: sb.grad_norm_clip([x, row], 0.5)
    yield "grad_norm_clip out", [y, bias], lambda: sb.grad_norm_clip([x, row], 0.5, out=[y, bias])
    yield "GradNormClip", [x, row], sb.GradNormClip([x, row], 0.5)
    yield "GradNormClip out", [y, bias], sb.GradNormClip([x, row], 0.5, out=[y, bias])


def test_writes_raise_the_version(sb):
    for what, written, call in calls(sb):
        before = [t._version for t in written]
        call()
        assert all(t._version > v for t, v in zip(written, before)), what


def test_what_is_only_read_keeps_its_version(sb):
    x, y, row = heads(0), heads(1), torch.ones(16, device="cuda")
    f, _ = sb.rotary_frequencies(16)
    p = torch.arange(5, device="cuda")
    read = (x, y, row, f, p)
    before = [t._version for t in read]
    sb.layer_norm(x, row, row)
    sb.layer_norm_backward(y, x, row)
    sb.rotary(x, p, f, k=y)
    sb.grad_norm([x, row])
    sb.grad_norm_clip([x, row], 1.0, out=[x.clone(), row.clone()])
    sb.GradNormClip([x, row], None)()
    assert [t._version for t in read] == before


def test_prepared_outputs_count_every_call(sb):
    """A prepared call writes its own output anew each time."""
    x, dy, row = heads(0), heads(1), torch.ones(16, device="cuda")
    f, _ = sb.rotary_frequencies(16)
    p = torch.arange(5, device="cuda")
    backward, turn, norm = sb.LayerNormBackward(dy, x, row), sb.Rotary(x, p, f, k=dy), sb.GradNormClip([x], None)
    for plan, outs in ((sb.LayerNorm(x, row), None), (backward, backward.out), (turn, turn.out), (norm, [norm.norm])):
        outs = [plan.out] if outs is None else outs
        plan()
        before = [t._version for t in outs]
        plan()
        assert all(t._version > v for t, v in zip(outs, before)), type(plan).__name__


def test_backward_through_an_overwritten_tensor_is_refused(sb):
    x = heads(0)
    w = torch.randn(16, 16, generator=torch.Generator().manual_seed(9)).cuda().requires_grad_()
    f, _ = sb.rotary_frequencies(16)
    p = torch.arange(5, device="cuda")
    for write in (lambda t: sb.layer_norm(t, out=t), lambda t: sb.rotary(t, p, f, out=t),
                  lambda t: sb.grad_norm_clip([t], 1e-3), lambda t: sb.layer_norm_backward(x, x, dx=t)):
        t = x.clone()
        loss = (t @ w).sum()  # saves t for w's gradient
        write(t)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_inference_tensors_are_taken(sb):
    with torch.inference_mode():
        x = heads(0)
        want = sb.layer_norm(x)
        assert torch.equal(sb.layer_norm(x, out=x), want)
        sb.grad_norm_clip([x], 1e-3)
