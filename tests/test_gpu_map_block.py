"""The feature-map operators together, as examples/vision_block.py trains with
them: every gradient of the block against torch.autograd on the same formulas
in 64 bits, and a few steps of training."""
import os
import sys

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block():
    import __graft_entry__
    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import vision_block
    torch.cuda.set_device(0)
    return vision_block


def plain(model, images, step, masks):
    """The block in torch operations on float64; masks: its two dropout factors."""
    n, _, s, _ = images.shape
    k, F = s // model.patch, torch.nn.functional
    w = {name: p.detach().double().requires_grad_(True) for name, p in model.named_parameters()}
    tokens = images.double().view(n, 3, k, model.patch, k, model.patch).permute(0, 2, 4, 1, 3, 5).reshape(n, k, k, -1)

    def resized(v, size):
        return F.interpolate(v.permute(0, 3, 1, 2), size=(size, size), mode="bilinear", align_corners=False).permute(0, 2, 3, 1)

    x = tokens @ w["embed"] + resized(w["table"], k)
    h = F.group_norm(x.permute(0, 3, 1, 2), model.groups, w["gamma"], w["beta"], 1e-5).permute(0, 2, 3, 1)
    h = F.silu(h) * masks[0]
    x = (h @ w["mix"]) * masks[1] + x
    return resized(x, 2 * k) @ w["out"], w


def test_gradients_of_the_block(block):
    import bilinear_image_resize_gb300 as rz
    torch.backends.cuda.matmul.allow_tf32 = False
    model = block.VisionBlock(patch=8, width=48, groups=6, p=0.2, table=5, dtype=torch.float32).cuda()
    g = torch.Generator(device="cuda").manual_seed(2)
    images = torch.randn((3, 3, 56, 56), device="cuda", generator=g)
    target = torch.randn((3, 14, 14, 3), device="cuda", generator=g)
    out = model(images, 4)
    (out - target).square().mean().backward()
    ones, masks = torch.ones((3, 7, 7, 48), device="cuda"), []
    for offset in (8, 9):
        m = torch.empty_like(ones)
        rz.map_dropout(ones, m, 0.2, model.seed, offset)
        masks.append(m.double())
    want, w = plain(model, images, 4, masks)
    (want - target.double()).square().mean().backward()
    # float32 against 64 bits: products of 192 and 48 terms and the sums over 147 to 588 pixels behind each gradient,
    # each within a few hundred units of its size
    assert float((out - want).abs().max()) <= 512 * 2.0 ** -24 * float(want.abs().max())
    for name, p in model.named_parameters():
        ref = w[name].grad
        assert float((p.grad - ref).norm()) <= 512 * 2.0 ** -24 * float(ref.norm()), name


def test_training_steps(block):
    losses = block.train(steps=12)
    assert all(b < a for a, b in zip(losses[:3], losses[1:4])) and losses[-1] < 0.8 * losses[0]
