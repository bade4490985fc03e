"""Fine-tuning steps of one transformer block over a clip's latent tokens.

The block predicts the noise in latents: layer norm, one projection to query,
key and value heads, a norm over each query and key head (in place of the packed
projection's views, no copy), rotary embedding by (frame, row, column), attention,
projection.  Its gradients are clipped by their global norm into the 32-bit ones
that the update takes.  Layer norm, rotary embedding and clipping are this
library's; matrix products and the softmax are torch's.

    python examples/latent_block_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Norm(torch.autograd.Function):
    """layer_norm with its gradient, for torch's autograd."""

    @staticmethod
    def forward(ctx, x, gamma, beta):
        import seam_blending_patch_amd as sb
        ctx.save_for_backward(x, gamma)
        return sb.layer_norm(x, gamma, beta)

    @staticmethod
    def backward(ctx, dy):
        import seam_blending_patch_amd as sb
        return sb.layer_norm_backward(dy.contiguous(), *ctx.saved_tensors)


class Turn(torch.autograd.Function):
    """rotary of query and key heads with its gradient."""

    @staticmethod
    def forward(ctx, q, k, positions, freqs, sections):
        import seam_blending_patch_amd as sb
        ctx.save_for_backward(positions, freqs)
        ctx.sections = sections
        return sb.rotary(q, positions, freqs, k=k, sections=sections, interleaved=True)

    @staticmethod
    def backward(ctx, dq, dk):
        import seam_blending_patch_amd as sb
        positions, freqs = ctx.saved_tensors
        dq, dk = sb.rotary_backward(dq.contiguous(), positions, freqs, k=dk.contiguous(), sections=ctx.sections,
                                    interleaved=True)
        return dq, dk, None, None, None


def weights(width: int, heads: int, dtype, device, seed: int = 0):
    """The block's parameters, in the order that block() takes them."""
    gen = torch.Generator().manual_seed(seed)
    d = width // heads
    shapes = [(width,), (width,), (width, 3 * width), (d,), (d,), (d,), (d,), (width, width)]
    made = [torch.randn(s, generator=gen) / s[0] ** 0.5 if len(s) == 2
            else torch.ones(s) if k in (0, 3, 5) else torch.zeros(s) for k, s in enumerate(shapes)]
    return [w.to(dtype).to(device).requires_grad_() for w in made]


def block(x, w, heads: int, positions, freqs, sections, norm=Norm.apply, turn=Turn.apply):
    """[tokens, width] -> [tokens, width]"""
    gamma, beta, w_qkv, q_gamma, q_beta, k_gamma, k_beta, w_out = w
    tokens, width = x.shape
    d = width // heads
    qkv = (norm(x, gamma, beta) @ w_qkv).view(tokens, 3, heads, d)
    q, k = norm(qkv[:, 0], q_gamma, q_beta), norm(qkv[:, 1], k_gamma, k_beta)
    q, k = turn(q, k, positions, freqs, sections)
    # attention in at least 32 bits, head by head: [heads, tokens, d]
    wide = torch.promote_types(x.dtype, torch.float32)
    q, k, v = (t.transpose(0, 1).to(wide).contiguous() for t in (q, k, qkv[:, 2]))
    scores = torch.bmm(q, k.transpose(1, 2).contiguous()) / d ** 0.5
    mixed = torch.bmm(torch.softmax(scores, -1), v).transpose(0, 1).reshape(tokens, width).to(x.dtype)
    return x + mixed @ w_out


def grid_positions(frames: int, rows: int, cols: int, device):
    """[3, tokens]: the frame, row and column of every latent token."""
    axes = [torch.arange(n, device=device) for n in (frames, rows, cols)]
    return torch.stack([a.flatten() for a in torch.meshgrid(*axes, indexing="ij")])


def main(steps: int = 20, width: int = 256, heads: int = 4, grid=(3, 10, 13), dtype=torch.bfloat16, rate: float = 4.0,
         max_norm: float = 0.02):
    import seam_blending_patch_amd as sb
    device = torch.device("cuda")
    w = weights(width, heads, dtype, device)
    masters = [p.detach().float() for p in w]
    grads32 = [torch.empty_like(m) for m in masters]
    positions = grid_positions(*grid, device)
    pairs = width // heads // 2
    sections = (pairs - 2 * (pairs // 3), pairs // 3, pairs // 3)
    freqs, _ = sb.rotary_frequencies(2 * pairs, sections=sections)
    gen = torch.Generator(device=device).manual_seed(1)
    latents = torch.randn(positions.shape[1], width, generator=gen, device=device)
    noise = torch.randn(latents.shape, generator=gen, device=device)
    x = (0.7 * latents + 0.7 * noise).to(dtype)
    history = []
    for step in range(steps):
        loss = (block(x, w, heads, positions, freqs, sections).float() - noise).square().mean()
        grads = torch.autograd.grad(loss, w)
        norm = sb.grad_norm_clip(grads, max_norm, out=grads32)
        with torch.no_grad():
            for p, m, g in zip(w, masters, grads32):
                m -= rate * g
                p.copy_(m)
        history.append((loss.item(), norm.item()))
        print(f"step {step}: loss {history[-1][0]:.4f}, gradient norm {history[-1][1]:.4f}", flush=True)
    return history


if __name__ == "__main__":
    main()
