"""The 64-bit forms that the feature-map kernels are held to, against things
that do not share their code: published vectors of the generator, torch's
own float64 group norm and bilinear resize, and differences of the forward
forms for the gradients."""
import numpy as np
import pytest

import map_reference as ref


def test_philox_published_vectors():
    # Random123's known answers of philox4x32 with 10 rounds
    assert ref.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert ref.philox([0xffffffff] * 4, [0xffffffff] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert ref.philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_drop_rate_and_scale():
    f = ref.drop_factor((40000,), 0.3, 11, 5)
    t = ref.threshold(0.3)
    assert set(np.unique(f)) == {0.0, 65536 / (65536 - t)}
    assert abs((f == 0).mean() - 0.3) < 5 * np.sqrt(0.21 / 40000)
    # a window of it is the same elements
    np.testing.assert_array_equal(f[1003:1100], ref.drop_factor((97,), 0.3, 11, 5, first=1003))
    assert np.all(ref.drop_factor((64,), 1.0, 1, 0) == 0) and np.all(ref.drop_factor((64,), 0.0, 1, 0) == 1)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_norm_against_torch(kind):
    import torch
    rng = np.random.default_rng(3)
    x, gamma, beta = rng.normal(1, 2, (2, 5, 7, 12)), rng.normal(1, 0.2, 12), rng.normal(0, 0.3, 12)
    y = ref.group_norm(x, 4, gamma, beta, kind, 1e-5, np.ones_like(x))[0]
    t = torch.nn.functional.group_norm(torch.from_numpy(x).permute(0, 3, 1, 2), 4, torch.from_numpy(gamma),
                                       torch.from_numpy(beta), 1e-5)
    t = {"none": lambda v: v, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[kind](t)
    np.testing.assert_allclose(y, t.permute(0, 2, 3, 1).numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("kind", ["none", "silu", "gelu"])
def test_norm_gradient_against_differences(kind):
    rng = np.random.default_rng(4)
    x, gamma, beta = rng.normal(0.5, 1.5, (2, 3, 4, 6)), rng.normal(1, 0.2, 6), rng.normal(0, 0.3, 6)
    factor, dy = ref.drop_factor(x.shape, 0.25, 9, 2), rng.normal(size=x.shape)

    def loss(x, gamma, beta):
        return (dy * ref.group_norm(x, 3, gamma, beta, kind, 1e-3, factor)[0]).sum()

    _, mean, rstd, _ = ref.group_norm(x, 3, gamma, beta, kind, 1e-3, factor)
    dx, dgamma, dbeta, _, _ = ref.group_norm_grad(dy, x, 3, gamma, beta, mean, rstd, kind, factor)
    h = 1e-5
    for _ in range(5):
        vx, vg, vb = rng.normal(size=x.shape), rng.normal(size=6), rng.normal(size=6)
        slope = (loss(x + h * vx, gamma + h * vg, beta + h * vb) - loss(x - h * vx, gamma - h * vg, beta - h * vb)) / (2 * h)
        assert abs(slope - ((dx * vx).sum() + (dgamma * vg).sum() + (dbeta * vb).sum())) < 1e-6 * (1 + abs(slope))


@pytest.mark.parametrize("geo", [(5, 7, 10, 14), (9, 4, 5, 3), (1, 6, 4, 1), (3, 3, 3, 3), (6, 5, 13, 9)])
def test_resize_against_torch_and_its_transpose(geo):
    import torch
    H, W, OH, OW = geo
    rng = np.random.default_rng(5)
    src, d = rng.normal(size=(2, H, W, 3)), rng.normal(size=(2, OH, OW, 3))
    out = ref.resize(src, OH, OW)
    t = torch.nn.functional.interpolate(torch.from_numpy(src).permute(0, 3, 1, 2), size=(OH, OW), mode="bilinear",
                                        align_corners=False).permute(0, 2, 3, 1).numpy()
    np.testing.assert_allclose(out, t, rtol=1e-11, atol=1e-12)
    assert abs((out * d).sum() - (src * ref.resize_grad(d, H, W)).sum()) < 1e-10
