"""The example's block: gradients through the library's operators against the
same block of plain 64-bit operations, and a few of its steps."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import transformer_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("latent_block_step",
                                                  os.path.join(ROOT, "examples", "latent_block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_norm(x, gamma, beta):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + 1e-6) * gamma + beta


def plain_turn(q, k, positions, freqs, sections):
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    angle = positions.t()[:, axis].double() * freqs
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    turned = []
    for x in (q, k):
        u, v = x[..., 0::2], x[..., 1::2]
        turned.append(torch.stack((u * c - v * s, u * s + v * c), -1).flatten(-2))
    return turned


def test_gradients_through_the_block(example):
    """fp32 on the GPU against 64 bits on the CPU.  Four products over 96 terms
    and two over 42, three norms and a softmax, forward and back: each product is
    off by at most 96 U of the sum of its terms' magnitudes, about 10 times its
    size here, so a gradient by some 12 * 96 * 10 U = 7e-4 of its norm in the
    worst case; the errors are random and a tenth of that is allowed."""
    import seam_blending_patch_amd as sb
    width, heads, sections = 96, 3, (6, 5, 5)
    grid = (2, 3, 7)
    w = example.weights(width, heads, torch.float32, "cuda", 3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(42, width, generator=gen)
    target = torch.randn(42, width, generator=gen)
    freqs, _ = sb.rotary_frequencies(32, sections=sections)
    positions = example.grid_positions(*grid, "cuda")
    y = example.block(x.cuda(), w, heads, positions, freqs, sections)
    got = torch.autograd.grad((y - target.cuda()).square().mean(), w)
    w64 = [p.detach().cpu().double().requires_grad_() for p in w]
    y64 = example.block(x.double(), w64, heads, positions.cpu(), freqs.cpu(), sections, plain_norm, plain_turn)
    want = torch.autograd.grad((y64 - target.double()).square().mean(), w64)
    assert np.linalg.norm(ref.f64(y) - ref.f64(y64)) <= 7e-5 * np.linalg.norm(ref.f64(y64))
    for k, (g, h) in enumerate(zip(got, want)):
        assert np.linalg.norm(ref.f64(g) - ref.f64(h)) <= 7e-5 * np.linalg.norm(ref.f64(h)), f"parameter {k}"


def test_steps_learn(example):
    history = example.main(steps=6)
    losses, norms = zip(*history)
    assert losses[-1] < losses[0] and all(np.isfinite(norms))
