"""Dropout from a counter against the 64-bit form: exact masks, whatever the
layout, the vector width and the split of the map."""
import numpy as np
import pytest

import map_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def values(shape, dtype, seed):
    x = np.random.default_rng(seed).normal(size=shape)
    x[np.abs(x) < 1e-3] = 1e-3       # no zero of its own: the mask shows
    return ref.host(torch.from_numpy(x).to(TYPES[dtype]))


def check(rz, shape, dtype, p, residual, layout={}, seed=(1 << 40) + 9, offset=(7 << 32) + 5, stream=None):
    x, r = values(shape, dtype, 1), values(shape, dtype, 2)
    xv, _ = ref.device_map(x, dtype, **layout)
    rv = ref.device_map(r, dtype, **layout)[0] if residual else None
    yv, flat = ref.device_map(np.zeros(shape), dtype, fill=-3.0, **layout)
    rz.map_dropout(xv, yv, p, seed, offset, residual=rv, stream=stream)
    torch.cuda.synchronize()
    factor = ref.drop_factor(shape, p, seed, offset)
    want = x * factor + (r if residual else 0)
    # the scale, the product and the sum each round once
    err = ref.U * (2 * np.abs(x * factor) + np.abs(want))
    got = ref.host(yv)
    if not residual:
        np.testing.assert_array_equal(got == 0, factor == 0)
    assert np.all(np.abs(got - want) <= ref.stored(want, err, dtype))
    assert ref.outside_untouched(flat, yv, -3.0)
    return yv


SHAPES = [(1, 1, 1, 1), (1, 1, 1, 7), (1, 1, 3, 5), (2, 3, 4, 8), (3, 5, 7, 24), (1, 61, 1, 200), (2, 9, 11, 3)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(rz, shape, dtype, residual):
    check(rz, shape, dtype, 0.3, residual)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("p", [0.0, 1e-6, 1 / 65536, 0.5, 65535 / 65536, 1.0])
def test_rates(rz, dtype, p):
    check(rz, (2, 6, 5, 16), dtype, p, True)
    check(rz, (1, 6, 5, 16), dtype, p, False)


@pytest.mark.parametrize("layout", [dict(pad=8), dict(pad=16, gap=8), dict(gap=40), dict(offset=1), dict(pad=3),
                                    dict(pad=4, offset=4)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [16, 5])
def test_layouts_keep_the_mask(rz, layout, dtype, C):
    a = check(rz, (2, 5, 7, C), dtype, 0.4, True, layout)
    b = check(rz, (2, 5, 7, C), dtype, 0.4, True)
    assert torch.equal(a, b)


def test_any_shape_of_packed_elements(rz):
    x = values((2, 3, 5, 8), "f32", 3)
    want = ref.drop_factor((240,), 0.5, 1, 0) != 0
    for shape in [(240,), (30, 8), (2, 3, 40), (2, 3, 5, 8), (2, 3, 5, 4, 2), (1, 240)]:
        t = torch.from_numpy(x.reshape(shape)).float().cuda()
        y = torch.empty_like(t)
        rz.map_dropout(t, y, 0.5, 1)
        np.testing.assert_array_equal(ref.host(y).reshape(-1) != 0, want)
    rz.map_dropout(torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), 0.5, 1)
    rz.map_dropout(torch.empty((3, 0), device="cuda"), torch.empty((3, 0), device="cuda"), 0.5, 1)
    s = torch.ones((), device="cuda")
    rz.map_dropout(s, s, 0.0, 1)


def test_in_place_and_onto_the_residual(rz):
    x, r = (torch.from_numpy(values((2, 4, 4, 16), "f32", k)).float().cuda() for k in (4, 5))
    want = torch.empty_like(x)
    rz.map_dropout(x, want, 0.3, 6, 7, residual=r)
    a, b = x.clone(), r.clone()
    rz.map_dropout(a, a, 0.3, 6, 7, residual=r)
    rz.map_dropout(x, b, 0.3, 6, 7, residual=b)
    assert torch.equal(a, want) and torch.equal(b, want)


def test_dropped_elements_are_zero_whatever_they_held(rz):
    x = torch.full((1, 8, 8, 64), float("nan"), device="cuda")
    x[..., ::2] = float("inf")
    y = torch.empty_like(x)
    rz.map_dropout(x, y, 1.0, 3)
    assert bool((y == 0).all())
    rz.map_dropout(x, y, 0.5, 3)
    kept = torch.from_numpy(ref.drop_factor((1, 8, 8, 64), 0.5, 3, 0) != 0).cuda()
    assert bool((y[~kept] == 0).all()) and not bool(y[kept].isfinite().any())


def test_gradient_is_the_same_mask(rz):
    # y is linear in x, so a difference of the forward along v is the gradient's product with v
    x, v, dy = (torch.from_numpy(values((2, 7, 3, 24), "f32", k)).float().cuda() for k in (6, 7, 8))
    y0, y1, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    rz.map_dropout(x, y0, 0.25, 11, 12, residual=v)
    rz.map_dropout(x + v, y1, 0.25, 11, 12, residual=v)
    rz.map_dropout(dy, dx, 0.25, 11, 12)
    moved, product = ((y1 - y0).double() * dy.double()).sum(), (dx.double() * v.double()).sum()
    size = (dy.double() * v.double()).abs().sum()
    assert abs(float(moved - product)) <= 16 * ref.U * 4 * float(size)


def test_the_mask_of_the_norm(rz):
    # a constant map with a unit shift: what the norm's own dropout leaves is this mask
    x = torch.ones((2, 5, 5, 16), device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    rz.map_group_norm(x, y, 4, torch.ones(16, device="cuda"), torch.ones(16, device="cuda"), drop=(0.4, 21, 22))
    rz.map_dropout(x, z, 0.4, 21, 22)
    assert torch.equal(y, z)


def test_elements_past_32_bits(rz):
    n = (1 << 32) + 4096
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda").view(-1, 4096)
    rz.map_dropout(x, x, 0.5, 31, 32)
    for first in (0, (1 << 31) - 2048, (1 << 32) - 2048, n - 4096):
        want = ref.drop_factor((4096,), 0.5, 31, 32, first=first)
        np.testing.assert_array_equal(ref.host(x.view(-1)[first:first + 4096]), want)


def test_on_another_stream(rz):
    s = torch.cuda.Stream()
    a = check(rz, (2, 5, 7, 24), "bf16", 0.3, True, stream=s)
    b = check(rz, (2, 5, 7, 24), "bf16", 0.3, True)
    assert torch.equal(a, b)


def test_refusals(rz):
    x = torch.zeros((2, 4, 4, 8), device="cuda")
    flat = torch.zeros(264, device="cuda")
    for call in (lambda: rz.map_dropout(x, torch.empty_like(x), -0.1, 0),
                 lambda: rz.map_dropout(x, torch.empty_like(x), 1.5, 0),
                 lambda: rz.map_dropout(x, torch.empty_like(x), float("nan"), 0),
                 lambda: rz.map_dropout(flat[:256], flat[8:], 0.1, 0),
                 lambda: rz.map_dropout(x.view(-1), flat[:256], 0.1, 0, residual=flat[8:])):
        with pytest.raises(rz.ResizeError) as e:
            call()
        assert e.value.code == rz.RZ_ERR_ARG
    for bad in (x.half(), x[:1], x.cpu()):
        with pytest.raises(ValueError):
            rz.map_dropout(x, bad, 0.1, 0)
        with pytest.raises(ValueError):
            rz.map_dropout(x, torch.empty_like(x), 0.1, 0, residual=bad)
    with pytest.raises(ValueError):
        rz.map_dropout(x.double(), x.double(), 0.1, 0)
