"""Group norm, attention and dropout run together in the spatial block: gradients
through the library's operators against the same block of plain 64-bit operations,
lengths, and a few of its steps."""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import pytest
import torch

import channels_ref
import transformer_ref as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "examples", name + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return load("spatial_block_step")


def plain_norm(x, gamma, beta, groups):
    h = x.reshape(x.shape[0], -1, groups, x.shape[-1] // groups)
    h = h - h.mean((1, 3), keepdim=True)
    z = (h / torch.sqrt((h * h).mean((1, 3), keepdim=True) + 1e-6)).reshape(x.shape) * gamma + beta
    return z / (1 + torch.exp(-z))


def plain_attend(qkv, lengths):
    out = []
    for b in range(qkv.shape[0]):
        n = qkv.shape[1] if lengths is None else int(lengths[b])
        q, k, v = qkv[b, :n].unbind(1)
        p = torch.softmax(torch.einsum("qhd,khd->hqk", q, k) / q.shape[-1] ** 0.5, -1)
        mixed = torch.einsum("hqk,khd->qhd", p, v)
        out.append(torch.cat((mixed, torch.zeros(qkv.shape[1] - n, *mixed.shape[1:], dtype=mixed.dtype))))
    return torch.stack(out)


def plain_drop(x, residual, p, state, site):
    words = channels_ref.words(x.numel(), int(state[0]), int(state[1]), site)
    keep = torch.from_numpy(words >= int(np.floor(p * 2.0 ** 32))).view(x.shape)
    return torch.where(keep, x / (1 - p), 0.0) + residual


@pytest.mark.parametrize("lengths", [None, [35, 14, 0]])
def test_gradients_through_the_block(example, lengths):
    """fp32 on the GPU against 64 bits on the CPU.  Two products over 96 terms and two
    over 35, a norm and a softmax, forward and back: each product is off by at most
    96 U of the sum of its terms' magnitudes, about 10 times its size here, so a
    gradient by some 8 * 96 * 10 U = 5e-4 of its norm in the worst case; the errors
    are random and a tenth of that is allowed."""
    w = example.weights(96, torch.float32, "cuda", 3)
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(3, 5, 7, 96, generator=gen)
    target = torch.randn(x.shape, generator=gen)
    state = torch.tensor([77, 5])
    on = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    xg = x.cuda().requires_grad_()
    y = example.block(xg, w, 8, 3, 0.2, state.cuda(), on, site=2)
    got = torch.autograd.grad((y - target.cuda()).square().mean(), [xg, *w])
    w64 = [p.detach().cpu().double().requires_grad_() for p in w]
    x64 = x.double().requires_grad_()
    y64 = example.block(x64, w64, 8, 3, 0.2, state, lengths, plain_norm, plain_attend, plain_drop, site=2)
    want = torch.autograd.grad((y64 - target.double()).square().mean(), [x64, *w64])
    assert np.linalg.norm(ref.f64(y) - ref.f64(y64)) <= 5e-5 * np.linalg.norm(ref.f64(y64))
    for k, (g, h) in enumerate(zip(got, want)):
        assert np.linalg.norm(ref.f64(g) - ref.f64(h)) <= 5e-5 * np.linalg.norm(ref.f64(h)), f"gradient {k}"


def test_a_captured_step_draws_new_masks(example):
    """forward, gradient and update in one graph: replays against eager steps from the
    same weights, the offset moved inside the graph"""
    def step(w, x, target, state, grads):
        loss = (example.block(x, w, 8, 4, 0.3, state) - target).square().mean()
        for g, new in zip(grads, torch.autograd.grad(loss, w)):
            g.copy_(new)
        state[1].add_(1)

    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(2, 6, 8, 64, generator=gen, device="cuda")
    target = x.roll(1, 1)
    w = example.weights(64, torch.float32, "cuda", 1)
    state, grads = torch.tensor([9, 0], device="cuda"), [torch.zeros_like(p) for p in w]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(w, x, target, state, grads)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(w, x, target, state, grads)
    other = example.weights(64, torch.float32, "cuda", 1)
    for turn in range(3):
        at = state.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert int(state[1]) == int(at[1]) + 1
        want = [torch.zeros_like(p) for p in other]
        step(other, x, target, at, want)
        torch.cuda.synchronize()
        # (the products are torch's: the same kernels, captured or not)
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), turn


def test_steps_run(example):
    history = example.main(steps=3)
    assert len(history) == 3 and np.isfinite(history).all()


def test_the_latent_block_attends_by_the_library():
    """the transformer block's attention against the plain one, on the GPU in 16 bits:
    results of the same inputs are a rounding of the probabilities and one of the
    results apart, 2^-8 of them each in the worst case"""
    m = load("latent_block_step")
    gen = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (torch.randn(390, 4, 64, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(3))
    a, b = m.Mix.apply(q, k, v).double(), m.plain_mix(q.float(), k.float(), v.float()).double()
    assert torch.linalg.norm(a - b) <= 2.0 ** -7 * torch.linalg.norm(b)
