"""The operators around attention together, as examples/vision_attention.py
trains with them: every gradient of the block against torch.autograd on the same
formulas in 64 bits, in each type, and a step captured in a graph."""
import os
import sys

import numpy as np
import pytest

import token_reference as tok
from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import vision_attention
    torch.cuda.set_device(0)
    torch.backends.cuda.matmul.allow_tf32 = False
    return vision_attention


def plain(m, images):
    """The block in torch operations on float64."""
    n, _, s, _ = images.shape
    k, F = s // m.patch, torch.nn.functional
    heads, dim = m.heads, m.dim
    w = {name: p.detach().double().requires_grad_(True) for name, p in m.named_parameters()}
    tokens = images.double().view(n, 3, k, m.patch, k, m.patch).permute(0, 2, 4, 1, 3, 5).reshape(n, k, k, -1)

    def norm(x, i):
        return F.group_norm(x.permute(0, 3, 1, 2), m.groups, w[f"gammas.{i}"], w[f"betas.{i}"], 1e-5).permute(0, 2, 3, 1)

    x = tokens @ w["embed"].T + F.interpolate(w["table"].permute(0, 3, 1, 2), size=(k, k), mode="bilinear").permute(0, 2, 3, 1)
    qkv = (norm(x, 0) @ w["qkv"].T).view(n, k, k, 3, heads, dim)
    at = torch.arange(k, dtype=torch.float64, device=images.device)
    rows = dim // 4
    t = torch.zeros((k, k, dim // 2), dtype=torch.float64, device=images.device)
    for j in range(rows):
        t[:, :, j] = at[:, None] * 100.0 ** (-j / rows)
    for j in range(dim // 2 - rows):
        t[:, :, rows + j] = at * 100.0 ** (-j / (dim // 2 - rows))
    c, sn = t.cos()[:, :, None], t.sin()[:, :, None]

    def turned(v, g):
        v = v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g
        a, b = v.chunk(2, -1)
        return torch.cat([a * c - b * sn, a * sn + b * c], -1).reshape(n, k * k, heads, dim).transpose(1, 2)

    q, key = turned(qkv[..., 0, :, :], w["gamma_q"]), turned(qkv[..., 1, :, :], w["gamma_k"])
    v = qkv[..., 2, :, :].reshape(n, k * k, heads, dim).transpose(1, 2)
    b = tok.buckets(k, k, min(4, m.side), m.side, max(k, 5))
    r, cc = (torch.from_numpy(np.ascontiguousarray(i)).long().to(images.device) for i in tok.pair_buckets(b, b, (k, k), (k, k)))
    scores = q @ key.transpose(2, 3) * dim ** -0.5 + w["bias"][r, cc].permute(2, 0, 1)
    h = (scores.softmax(-1) @ v).transpose(1, 2).reshape(n, k, k, heads * dim)
    x = h @ w["proj"].T + x
    h = norm(x, 1) @ w["up"].T + w["up_bias"]
    h = h * torch.special.ndtr(h)
    x = h @ w["down"].T + w["down_bias"] + x
    return x @ w["out"].T, w


@pytest.mark.parametrize("dtype, units", [(torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)])
@pytest.mark.parametrize("heads, dim, size", [(3, 16, 56), (2, 24, 40)])
def test_gradients_of_the_block(example, dtype, units, heads, dim, size):
    m = example.AttentionBlock(patch=8, heads=heads, dim=dim, groups=6, table=5, side=5, dtype=dtype).cuda()
    with torch.no_grad():
        # weights that the type holds, so that their rounding is no error, and biases and gammas that matter
        g = torch.Generator(device="cuda").manual_seed(3)
        for name, p in m.named_parameters():
            if p.dim() == 1:
                p += 0.2 * torch.randn(p.shape, device="cuda", generator=g)
            elif name != "bias":
                p.copy_(p.to(dtype).float())
    g = torch.Generator(device="cuda").manual_seed(2)
    images = torch.randn((3, 3, size, size), device="cuda", generator=g).to(dtype).float()
    out = m(images)
    target = torch.randn(out.shape, device="cuda", generator=g)
    # a sum that leaves the gradients of 16-bit values of about 1
    loss = (out - target).square().sum()
    loss.backward()
    want, w = plain(m, images)
    (want - target.double()).square().sum().backward()
    # In float32 each of the block's dozen operators adds some ten to a hundred units of random sign to what passes it: 512.  In 16 bits
    # every result is rounded by up to `units` of its size, 0.58 of that in the 2-norm, and a gradient passes about thirty such
    # roundings of random sign: a root of thirty of them, 3.2 units, which the norms and the softmax between may raise by their
    # condition, here a factor of up to five: 16 units.
    bound = (512 if dtype is torch.float32 else 16) * units
    assert float((out - want).norm()) <= bound * float(want.norm())
    for name, p in m.named_parameters():
        ref = w[name].grad
        assert float((p.grad - ref).norm()) <= bound * float(ref.norm()), (name, float((p.grad - ref).norm() / ref.norm()))


def test_runs(example):
    losses = example.train(steps=3)
    assert len(losses) == 3 and all(np.isfinite(losses))


def test_step_captured_in_a_graph(example):
    m = example.AttentionBlock(patch=8, heads=2, dim=32, groups=4, table=5, side=5).cuda()
    m.buckets = lambda k, b=m.buckets(5): b                       # made before the capture: a copy from host memory
    images = torch.randn((2, 3, 40, 40), device="cuda")
    params = list(m.parameters())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            grads = torch.autograd.grad(m(images).square().sum(), params)
        del grads
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = torch.autograd.grad(m(images).square().sum(), params)
    for seed in (1, 2):
        images.copy_(torch.randn(images.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        want = torch.autograd.grad(m(images).square().sum(), params)
        # the library's calls give the same bits; torch's products under a graph may take another workspace, not other kernels
        for a, b in zip(got, want):
            assert float((a.float() - b.float()).norm()) <= 2.0 ** -6 * float(b.float().norm())
