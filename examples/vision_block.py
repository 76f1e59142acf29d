"""A small vision model trained on resized frames, its block made of the
library's feature-map operators.

    uint8 frames -> resize + normalise (resize_fused) -> patches -> tokens
    + a learned position table resized to the tokens' grid (resize_map)
    -> group norm + SiLU + dropout -> product -> dropout + residual
    -> doubled (resize_map) -> product -> regression on the frame itself

    python examples/vision_block.py [--steps 20]

The products are torch.matmul.  Each operator's gradient is the library's own
call, joined to torch.autograd by the Functions below.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bilinear_image_resize_gb300 as rz                          # noqa: E402
from bilinear_image_resize_gb300.synth import NORM_MEAN, NORM_STD   # noqa: E402


class NormActDrop(torch.autograd.Function):
    """dropout(silu(group_norm(x))); drop: (p, seed, offset) or None."""

    @staticmethod
    def forward(ctx, x, gamma, beta, groups, drop):
        y = torch.empty_like(x)
        mean, rstd = (torch.empty((x.shape[0], groups), device=x.device) for _ in range(2))
        rz.map_group_norm(x, y, groups, gamma, beta, mean, rstd, act=rz.RZ_ACT_SILU, drop=drop)
        ctx.save_for_backward(x, gamma, beta, mean, rstd)
        ctx.groups, ctx.drop = groups, drop
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
        rz.map_group_norm_grad(dy.contiguous(), x, dx, ctx.groups, gamma, beta, mean, rstd, dgamma, dbeta,
                               act=rz.RZ_ACT_SILU, drop=ctx.drop)
        return dx, dgamma, dbeta, None, None


class DropAdd(torch.autograd.Function):
    """dropout(x) + residual; nothing of the mask is kept between the passes."""

    @staticmethod
    def forward(ctx, x, residual, drop):
        y = torch.empty_like(x)
        rz.map_dropout(x, y, *drop, residual=residual)
        ctx.drop = drop
        return y

    @staticmethod
    def backward(ctx, dy):
        dx = torch.empty_like(dy, memory_format=torch.contiguous_format)
        rz.map_dropout(dy.contiguous(), dx, *ctx.drop)
        return dx, dy, None


class ResizeAdd(torch.autograd.Function):
    """base + the bilinear resize of src to `size`; one source image serves every image of base."""

    @staticmethod
    def forward(ctx, src, base, size):
        n = src.shape[0] if base is None else base.shape[0]
        dst = torch.empty((n, *size, src.shape[3]), dtype=src.dtype if base is None else base.dtype, device=src.device)
        rz.resize_map(src, dst, base=base)
        ctx.shape, ctx.dtype, ctx.add = src.shape, src.dtype, base is not None
        return dst

    @staticmethod
    def backward(ctx, d):
        g = torch.empty(ctx.shape, dtype=ctx.dtype, device=d.device)
        rz.resize_map_grad(d.contiguous(), g)
        return g, d if ctx.add else None, None


class VisionBlock(torch.nn.Module):
    def __init__(self, patch: int = 16, width: int = 256, groups: int = 32, p: float = 0.1, table: int = 24,
                 seed: int = 0, dtype=torch.bfloat16):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return torch.nn.Parameter(torch.randn(shape, generator=g) * shape[0] ** -0.5)

        self.patch, self.groups, self.p, self.seed, self.dtype = patch, groups, p, seed, dtype
        self.embed, self.mix, self.out = weight(3 * patch * patch, width), weight(width, width), weight(width, 3)
        self.table = torch.nn.Parameter(0.02 * torch.randn((1, table, table, width), generator=g))
        self.gamma, self.beta = torch.nn.Parameter(torch.ones(width)), torch.nn.Parameter(torch.zeros(width))

    def forward(self, images, step: int):
        """images: float32 (N, 3, S, S); the doubled grid's (N, 2 S / patch, 2 S / patch, 3) in float32."""
        n, _, s, _ = images.shape
        k = s // self.patch
        tokens = images.view(n, 3, k, self.patch, k, self.patch).permute(0, 2, 4, 1, 3, 5).reshape(n, k, k, -1)
        x = tokens.to(self.dtype) @ self.embed.to(self.dtype)
        x = ResizeAdd.apply(self.table, x, (k, k))
        # the generator's offset counts calls: every step and place has a mask of its own
        h = NormActDrop.apply(x, self.gamma, self.beta, self.groups, (self.p, self.seed, 2 * step))
        h = h @ self.mix.to(self.dtype)
        x = DropAdd.apply(h, x, (self.p, self.seed, 2 * step + 1))
        x = ResizeAdd.apply(x, None, (2 * k, 2 * k))
        return (x @ self.out.to(self.dtype)).float()


def normalised(frames, size: int = 224):
    """uint8 (N, H, W, 3) frames resized to size x size and normalised, float32 (N, 3, size, size)."""
    n, h, w, _ = frames.shape
    out = torch.empty((n, 3, size, size), device=frames.device)
    with rz.resize_plan_create(h, w, size, size, rz.RZ_LINEAR) as plan:
        rz.resize_fused(plan, frames, out, rz.make_epilogue(rz.RZ_EPI_NORMALIZE_NCHW, mean=NORM_MEAN, std=NORM_STD))
    return out


def train(steps: int = 20, batch: int = 8, device: str = "cuda", rate: float = 5e-5):
    """Losses of `steps` steps of Adam on synthetic frames."""
    g = torch.Generator(device=device).manual_seed(1)
    frames = torch.randint(0, 256, (batch, 12, 20, 3), dtype=torch.uint8, device=device, generator=g)
    frames = frames.repeat_interleave(15, 1).repeat_interleave(16, 2)       # blocks of colour, 180 x 320
    images = normalised(frames)
    model = VisionBlock().to(device)
    grid = 2 * images.shape[2] // model.patch
    target = torch.nn.functional.adaptive_avg_pool2d(images, grid).permute(0, 2, 3, 1)
    adam, losses = torch.optim.Adam(model.parameters(), lr=rate), []
    for step in range(steps):
        loss = (model(images, step) - target).square().mean()
        adam.zero_grad(set_to_none=True)
        loss.backward()
        adam.step()
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    a.add_argument("--steps", type=int, default=20)
    for i, loss in enumerate(train(a.parse_args().steps)):
        print(f"step {i}: loss {loss:.4f}")
