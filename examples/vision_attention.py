"""An attention block trained on resized frames, made of the library's operators
around attention.

    uint8 frames -> resize + normalise (resize_fused) -> patches
    -> product (map_linear) + a learned position table resized to the grid (resize_map)
    -> group norm -> product to queries, keys and values (map_linear)
    -> norm of queries and keys, turned by row and column (map_qk_norm)
    -> scores + relative position bias (map_position_bias) -> softmax -> values
    -> product added to the block's input (map_linear)
    -> group norm -> product with GELU -> product, added again (map_linear)
    -> regression on the frame itself

    python examples/vision_attention.py [--steps 20]

The products of queries and keys, and of the softmax and the values, are
torch.matmul.  Each operator's gradient is the library's own call, joined to
torch.autograd by the Functions below.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for p in (os.path.dirname(HERE), HERE):
    if p not in sys.path:
        sys.path.insert(0, p)

import bilinear_image_resize_gb300 as rz                          # noqa: E402
from vision_block import ResizeAdd, normalised                    # noqa: E402

BASE = 100.0        # of the position rotation: a grid's side is far below a turn of the slowest pair


class Linear(torch.autograd.Function):
    """act(x weight^T + bias) + residual."""

    @staticmethod
    def forward(ctx, x, weight, bias, residual, act):
        x = x.contiguous()
        y = x.new_empty((*x.shape[:3], weight.shape[0]))
        pre = torch.empty_like(y) if act != rz.RZ_ACT_NONE else None
        rz.map_linear(x, y, weight, bias, residual=residual, pre=pre, act=act)
        ctx.save_for_backward(x, weight, pre)
        ctx.act, ctx.biased, ctx.added = act, bias is not None, residual is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, pre = ctx.saved_tensors
        dx, dw = torch.empty_like(x), torch.empty_like(weight)
        db = torch.empty(weight.shape[0], device=x.device) if ctx.biased else None
        rz.map_linear_grad(dy.contiguous(), x, weight, dx, dw, db, pre=pre, act=ctx.act)
        return dx, dw, db, dy if ctx.added else None, None


class GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, groups):
        y = torch.empty_like(x)
        mean, rstd = (torch.empty((x.shape[0], groups), device=x.device) for _ in range(2))
        rz.map_group_norm(x, y, groups, gamma, beta, mean, rstd)
        ctx.save_for_backward(x, gamma, beta, mean, rstd)
        ctx.groups = groups
        return y

    @staticmethod
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
        rz.map_group_norm_grad(dy.contiguous(), x, dx, ctx.groups, gamma, beta, mean, rstd, dgamma, dbeta)
        return dx, dgamma, dbeta, None


class QkNorm(torch.autograd.Function):
    """Queries and keys out of (N, H, W, 3 E), normed and turned, (N, H, W, 2 E), and the values as they are."""

    @staticmethod
    def forward(ctx, qkv, gamma_q, gamma_k, heads, dim):
        e = heads * dim
        qk = qkv.new_empty((*qkv.shape[:3], 2 * e))
        rz.map_qk_norm(qkv, qk, heads, heads, dim, gamma_q, gamma_k, base=BASE, row_pairs=dim // 4)
        ctx.save_for_backward(qkv, gamma_q, gamma_k)
        ctx.heads, ctx.dim = heads, dim
        return qk, qkv[..., 2 * e:]

    @staticmethod
    def backward(ctx, dqk, dv):
        qkv, gamma_q, gamma_k = ctx.saved_tensors
        dqkv, dq, dk = torch.empty_like(qkv), torch.empty_like(gamma_q), torch.empty_like(gamma_k)
        # the values' channels are not touched by the operator: their gradient goes there
        dqkv[..., dqk.shape[-1]:] = dv
        rz.map_qk_norm_grad(dqk.contiguous(), qkv, dqkv, ctx.heads, ctx.heads, ctx.dim, gamma_q, gamma_k, dq, dk, base=BASE,
                            row_pairs=ctx.dim // 4)
        return dqkv, dq, dk, None, None


class PositionBias(torch.autograd.Function):
    """scores + the table's value for every query and key."""

    @staticmethod
    def forward(ctx, scores, table, rows, cols, grid):
        out = torch.empty_like(scores, memory_format=torch.contiguous_format)
        rz.map_position_bias(table, rows, cols, out, grid, grid, scores=scores.contiguous())
        ctx.save_for_backward(rows, cols)
        ctx.grid, ctx.shape = grid, table.shape
        return out

    @staticmethod
    def backward(ctx, d):
        rows, cols = ctx.saved_tensors
        dtable = torch.empty(ctx.shape, device=d.device)
        rz.map_position_bias_grad(d.contiguous(), rows, cols, dtable, ctx.grid, ctx.grid)
        return d, dtable, None, None, None


class AttentionBlock(torch.nn.Module):
    def __init__(self, patch: int = 16, heads: int = 4, dim: int = 64, groups: int = 32, table: int = 24, side: int = 6, seed: int = 0,
                 dtype=torch.bfloat16):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        width = heads * dim

        def weight(out, into):
            return torch.nn.Parameter(torch.randn((out, into), generator=g) * into ** -0.5)

        def vector(n, value):
            return torch.nn.Parameter(torch.full((n,), float(value)))

        self.patch, self.heads, self.dim, self.groups, self.side, self.dtype = patch, heads, dim, groups, side, dtype
        self.embed, self.qkv, self.proj = weight(width, 3 * patch * patch), weight(3 * width, width), weight(width, width)
        self.up, self.down, self.out = weight(4 * width, width), weight(width, 4 * width), weight(3, width)
        self.up_bias, self.down_bias = vector(4 * width, 0), vector(width, 0)
        self.table = torch.nn.Parameter(0.02 * torch.randn((1, table, table, width), generator=g))
        self.bias = torch.nn.Parameter(0.02 * torch.randn((2 * side - 1, 2 * side - 1, heads), generator=g))
        self.gammas = torch.nn.ParameterList([vector(width, 1), vector(width, 1)])
        self.betas = torch.nn.ParameterList([vector(width, 0), vector(width, 0)])
        self.gamma_q, self.gamma_k = vector(dim, 1), vector(dim, 1)

    def buckets(self, k):
        """Buckets of the offsets of an axis of k places: four by themselves, further ones share."""
        b = rz.map_position_buckets(k, k, exact=min(4, self.side), side=self.side, reach=max(k, 5))
        return torch.from_numpy(b).to(self.bias.device)

    def linear(self, x, weight, bias=None, residual=None, act=rz.RZ_ACT_NONE):
        return Linear.apply(x, weight.to(self.dtype), bias, residual, act)

    def forward(self, images):
        """images: float32 (N, 3, S, S); (N, S / patch, S / patch, 3) in float32."""
        n, _, s, _ = images.shape
        k, heads, dim = s // self.patch, self.heads, self.dim
        tokens = images.view(n, 3, k, self.patch, k, self.patch).permute(0, 2, 4, 1, 3, 5).reshape(n, k, k, -1)
        x = ResizeAdd.apply(self.table, self.linear(tokens.to(self.dtype), self.embed), (k, k))
        h = GroupNorm.apply(x, self.gammas[0], self.betas[0], self.groups)
        qk, v = QkNorm.apply(self.linear(h, self.qkv), self.gamma_q, self.gamma_k, heads, dim)
        q, key, v = (t.reshape(n, k * k, heads, dim).transpose(1, 2) for t in (*qk.split(heads * dim, -1), v))
        scores = (q @ key.transpose(2, 3)) * dim ** -0.5
        at = self.buckets(k)
        scores = PositionBias.apply(scores, self.bias, at, at, (k, k))
        h = (torch.softmax(scores, -1) @ v).transpose(1, 2).reshape(n, k, k, heads * dim)
        x = self.linear(h, self.proj, residual=x)
        h = GroupNorm.apply(x, self.gammas[1], self.betas[1], self.groups)
        h = self.linear(h, self.up, self.up_bias, act=rz.RZ_ACT_GELU)
        x = self.linear(h, self.down, self.down_bias, residual=x)
        return self.linear(x, self.out).float()


def train(steps: int = 20, batch: int = 8, device: str = "cuda", rate: float = 1e-4):
    """Losses of `steps` steps of Adam on synthetic frames."""
    g = torch.Generator(device=device).manual_seed(1)
    frames = torch.randint(0, 256, (batch, 12, 20, 3), dtype=torch.uint8, device=device, generator=g)
    frames = frames.repeat_interleave(15, 1).repeat_interleave(16, 2)       # blocks of colour, 180 x 320
    images = normalised(frames)
    model = AttentionBlock().to(device)
    target = torch.nn.functional.adaptive_avg_pool2d(images, images.shape[2] // model.patch).permute(0, 2, 3, 1)
    adam, losses = torch.optim.Adam(model.parameters(), lr=rate), []
    for _ in range(steps):
        loss = (model(images) - target).square().mean()
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
