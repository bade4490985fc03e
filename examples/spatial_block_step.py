"""Fine-tuning steps of a spatial attention block, as VAEs and U-Nets have them.

The block works on channels-last activations [N, height, width, channels]: group
norm with SiLU, a projection to query, key and value heads, attention of every
position to all of its image (or, of its first rows, where images of a batch are
of unlike heights), a projection, dropout and the residual.  Its positions are
attention's tokens as they lie: nothing is transposed.  The parameters' gradients
are clipped by their global norm.  Group norm, attention, dropout and clipping are
this library's; matrix products are torch's.

    python examples/spatial_block_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class NormAct(torch.autograd.Function):
    """group_norm with SiLU, with its gradient, for torch's autograd."""

    @staticmethod
    def forward(ctx, x, gamma, beta, groups):
        import seam_blending_patch_amd as sb
        y, stats = sb.group_norm(x, groups, gamma, beta, activation="silu", return_stats=True)
        ctx.save_for_backward(x, gamma, beta, stats)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        import seam_blending_patch_amd as sb
        x, gamma, beta, stats = ctx.saved_tensors
        return (*sb.group_norm_backward(dy.contiguous(), x, ctx.groups, stats, gamma, beta, activation="silu"), None)


class Attend(torch.autograd.Function):
    """attention of packed heads [B, T, 3, heads, D], with its gradient written into
    one packed tensor."""

    @staticmethod
    def forward(ctx, qkv, lengths):
        import seam_blending_patch_amd as sb
        q, k, v = qkv.unbind(2)
        out, lse = sb.attention(q, k, v, query_lengths=lengths, key_lengths=lengths, return_lse=True)
        ctx.save_for_backward(qkv, out, lse, lengths)
        return out

    @staticmethod
    def backward(ctx, dout):
        import seam_blending_patch_amd as sb
        qkv, out, lse, lengths = ctx.saved_tensors
        grad = torch.empty_like(qkv)
        dq, dk, dv = grad.unbind(2)
        sb.attention_backward(dout.contiguous(), *qkv.unbind(2), out, lse, query_lengths=lengths, key_lengths=lengths,
                              dq=dq, dk=dk, dv=dv)
        return grad, None


class DropAdd(torch.autograd.Function):
    """residual + dropout, with its gradient."""

    @staticmethod
    def forward(ctx, x, residual, p, state, site):
        import seam_blending_patch_amd as sb
        ctx.save_for_backward(state.clone())  # (the step moves the offset on)
        ctx.p, ctx.site = p, site
        return sb.dropout(x, p, state, site=site, residual=residual)

    @staticmethod
    def backward(ctx, dy):
        import seam_blending_patch_amd as sb
        return sb.dropout_backward(dy.contiguous(), ctx.p, *ctx.saved_tensors, site=ctx.site), dy, None, None, None


def weights(channels: int, dtype, device, seed: int = 0):
    """The block's parameters, in the order that block() takes them."""
    gen = torch.Generator().manual_seed(seed)
    shapes = [(channels,), (channels,), (channels, 3 * channels), (channels, channels)]
    made = [torch.randn(s, generator=gen) / s[0] ** 0.5 if len(s) == 2 else torch.ones(s) if k == 0 else torch.zeros(s)
            for k, s in enumerate(shapes)]
    return [w.to(dtype).to(device).requires_grad_() for w in made]


def block(x, w, groups: int, heads: int, p: float, state, lengths=None, norm=NormAct.apply, attend=Attend.apply,
          drop=DropAdd.apply, site: int = 0):
    """[N, height, width, channels] -> the same; lengths: int32 [N] positions of each image, or None."""
    gamma, beta, w_qkv, w_out = w
    n, c = x.shape[0], x.shape[-1]
    qkv = (norm(x, gamma, beta, groups) @ w_qkv).view(n, -1, 3, heads, c // heads)
    return drop((attend(qkv, lengths).reshape(n, -1, c) @ w_out).view(x.shape), x, p, state, site)


def main(steps: int = 20, channels: int = 320, groups: int = 32, heads: int = 8, size=(4, 24, 32), p: float = 0.1,
         dtype=torch.bfloat16, rate: float = 0.5, max_norm: float = 1.0):
    import seam_blending_patch_amd as sb
    device = torch.device("cuda")
    w = weights(channels, dtype, device)
    masters = [q.detach().float() for q in w]
    grads32 = [torch.empty_like(m) for m in masters]
    state = torch.tensor([1234, 0], device=device)  # the generator's seed and the step's offset
    gen = torch.Generator(device=device).manual_seed(1)
    x = torch.randn(*size, channels, generator=gen, device=device).to(dtype)
    target = x.float().roll(1, 2)
    history = []
    for step in range(steps):
        loss = (block(x, w, groups, heads, p, state).float() - target).square().mean()
        grads = torch.autograd.grad(loss, w)
        norm = sb.grad_norm_clip(grads, max_norm, out=grads32)
        state[1] += 1
        with torch.no_grad():
            for q, m, g in zip(w, masters, grads32):
                m -= rate * g
                q.copy_(m)
        history.append((loss.item(), norm.item()))
        print(f"step {step}: loss {history[-1][0]:.4f}, gradient norm {history[-1][1]:.4f}", flush=True)
    return history


if __name__ == "__main__":
    main()
