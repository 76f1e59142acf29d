"""Group norm with an activation and dropout on channels-last maps, and its
gradient, against the 64-bit forms."""
import ctypes

import numpy as np
import pytest

import map_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ACTS = {"none": 0, "silu": 1, "gelu": 2}


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def params(C, seed):
    rng = np.random.default_rng(seed)
    return (rng.normal(1, 0.3, C).astype(np.float32).astype(np.float64),
            rng.normal(0, 0.3, C).astype(np.float32).astype(np.float64))


def features(shape, dtype, seed, spreadv=1.0, offset=0.5):
    """What a convolution leaves: an offset and a scale for each channel; rounded to the type."""
    rng = np.random.default_rng(seed)
    C = shape[-1]
    x = rng.normal(size=shape) * (0.5 + rng.random(C)) * spreadv + offset * rng.normal(size=C)
    return ref.host(torch.from_numpy(x).to({"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]))


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).float().cuda()


def check_forward(rz, x, G, dtype, kind, p=0.0, layout={}, eps=1e-5, affine=True, stream=None, seed=5):
    N, H, W, C = x.shape
    gamma, beta = params(C, seed)
    if not affine:
        gamma, beta = np.ones(C), np.zeros(C)
    factor = ref.drop_factor(x.shape, p, 77, 3)
    xv, _ = ref.device_map(x, dtype, **layout)
    yv, flat = ref.device_map(np.zeros_like(x), dtype, fill=-3.0, **layout)
    yv.fill_(7.0)
    mean, rstd = (torch.full((N, G), 9.0, device="cuda") for _ in range(2))
    rz.map_group_norm(xv, yv, G, cuda(gamma) if affine else None, cuda(beta) if affine else None, mean, rstd,
                      act=ACTS[kind], eps=eps, drop=(p, 77, 3) if p else None, stream=stream)
    torch.cuda.synchronize()
    eps = float(np.float32(eps))
    want, wm, wr, _ = ref.group_norm(x, G, gamma, beta, kind, eps, factor)
    ty, tm, tr = ref.norm_bounds(x, G, gamma, beta, kind, eps, factor, dtype)
    assert np.all(np.abs(ref.host(mean) - wm) <= tm)
    assert np.all(np.abs(ref.host(rstd) - wr) <= tr)
    err = np.abs(ref.host(yv) - want)
    assert np.all(err <= ty), float((err / np.maximum(ty, 1e-30)).max())
    assert ref.outside_untouched(flat, yv, -3.0)
    return yv


def check_gradient(rz, x, G, dtype, kind, p=0.0, layout={}, eps=1e-5, affine=True, stream=None, seed=6):
    N, H, W, C = x.shape
    gamma, beta = params(C, seed)
    if not affine:
        gamma, beta = np.ones(C), np.zeros(C)
    factor = ref.drop_factor(x.shape, p, 78, 1 << 40)
    dy = features(x.shape, dtype, seed + 1, offset=0.1)
    _, mean, rstd, _ = ref.group_norm(x, G, gamma, beta, kind, eps, factor)
    mean, rstd = cuda(mean), cuda(rstd)
    xv, _ = ref.device_map(x, dtype, **layout)
    dv, _ = ref.device_map(dy, dtype, **layout)
    ov, flat = ref.device_map(np.zeros_like(x), dtype, fill=-3.0, **layout)
    dgamma, dbeta = (torch.full((C,), 9.0, device="cuda") for _ in range(2))
    rz.map_group_norm_grad(dv, xv, ov, G, cuda(gamma) if affine else None, cuda(beta) if affine else None, mean, rstd,
                           dgamma, dbeta, act=ACTS[kind], eps=eps, drop=(p, 78, 1 << 40) if p else None, stream=stream)
    torch.cuda.synchronize()
    args = (dy, x, G, gamma, beta, ref.host(mean), ref.host(rstd), kind, factor)
    want, wg, wb, _, _ = ref.group_norm_grad(*args)
    tx, tg, tb = ref.grad_bounds(*args, dtype)
    assert np.all(np.abs(ref.host(dgamma) - wg) <= tg)
    assert np.all(np.abs(ref.host(dbeta) - wb) <= tb)
    err = np.abs(ref.host(ov) - want)
    assert np.all(err <= tx), float((err / np.maximum(tx, 1e-30)).max())
    assert ref.outside_untouched(flat, ov, -3.0)


# one value a group; one pixel; rows of one; widths that fill no vector; groups
# that end inside a vector; more vectors of channels than a block has threads
SHAPES = [((1, 1, 1, 8), 2), ((2, 1, 1, 3), 3), ((2, 7, 5, 24), 8), ((1, 9, 1, 30), 5), ((3, 13, 17, 96), 8),
          ((2, 20, 31, 320), 32), ((1, 3, 5, 4224), 11), ((1, 64, 65, 16), 1), ((5, 12, 12, 64), 64), ((1, 1, 900, 40), 4)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape, G", SHAPES)
def test_forward(rz, shape, G, dtype):
    check_forward(rz, features(shape, dtype, 1), G, dtype, "silu")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape, G", SHAPES)
def test_gradient(rz, shape, G, dtype):
    check_gradient(rz, features(shape, dtype, 2), G, dtype, "silu")


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("p", [0.0, 0.1, 0.6])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [48, 21])
def test_activations_and_dropout(rz, kind, p, dtype, C):
    x = features((2, 9, 11, C), dtype, 3)
    check_forward(rz, x, 3, dtype, kind, p)
    check_gradient(rz, x, 3, dtype, kind, p)


# padded rows, gaps between images, starts that no vector is aligned to
LAYOUTS = [dict(pad=16), dict(gap=64), dict(pad=8, gap=24), dict(offset=1), dict(pad=4, offset=4), dict(pad=1)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_layouts(rz, layout, dtype):
    x = features((2, 11, 13, 32), dtype, 4)
    check_forward(rz, x, 4, dtype, "silu", 0.2, layout)
    check_gradient(rz, x, 4, dtype, "silu", 0.2, layout)


@pytest.mark.parametrize("shape, G", [((1, 150, 170, 32), 8), ((2, 96, 100, 128), 32), ((1, 300, 260, 8), 2),
                                      ((9, 40, 40, 72), 9)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_larger_images(rz, shape, G, dtype):
    x = features(shape, dtype, 5)
    check_forward(rz, x, G, dtype, "gelu")
    check_gradient(rz, x, G, dtype, "silu")


def test_without_scale_and_shift(rz):
    x = features((2, 6, 7, 32), "bf16", 6)
    check_forward(rz, x, 8, "bf16", "none", affine=False)
    check_gradient(rz, x, 8, "bf16", "none", affine=False)


@pytest.mark.parametrize("offset", [300.0, -20000.0])
@pytest.mark.parametrize("first", [0.0, 1.0])
def test_mean_far_above_the_deviation(rz, offset, first):
    # deviations survive whatever the mean, a first pixel unlike the others among them
    rng = np.random.default_rng(7)
    x = (rng.normal(size=(2, 30, 30, 32)) + offset)
    x[:, 0, 0] *= first
    x = x.astype(np.float32).astype(np.float64)
    check_forward(rz, x, 4, "f32", "none")


def test_constant_groups(rz):
    x = np.full((1, 8, 8, 16), 3.0)
    y = check_forward(rz, x, 4, "f32", "silu")
    gamma, beta = params(16, 5)
    # the mean is within a unit of 3, and 1 / sqrt(eps) = 316 scales what that leaves: 316 2^-22 1.7 (gamma) 1.1 (slope)
    np.testing.assert_allclose(ref.host(y)[0, 0, 0], ref.act(beta, "silu")[0], rtol=1e-5, atol=2e-4)


def test_not_a_number_stays_in_its_group(rz):
    x = features((2, 10, 10, 32), "f32", 8)
    bad = x.copy()
    bad[0, 3, 4, 9], bad[1, 2, 2, 30] = np.nan, np.inf
    outs = []
    for v in (x, bad):
        xv, _ = ref.device_map(v, "f32")
        y = torch.empty_like(xv)
        rz.map_group_norm(xv, y, 4, act=1)
        outs.append(ref.host(y))
    hit = np.zeros((2, 10, 10, 32), bool)
    hit[0, :, :, 8:16] = hit[1, :, :, 24:32] = True
    assert np.all(np.isnan(outs[1][hit]))
    np.testing.assert_array_equal(outs[0][~hit], outs[1][~hit])


def test_everything_dropped(rz):
    x = features((1, 4, 4, 16), "f32", 9)
    x[0, 0, 0, 0] = np.nan
    xv, _ = ref.device_map(x, "f32")
    y = torch.full_like(xv, 5.0)
    rz.map_group_norm(xv, y, 2, act=2, drop=(1.0, 1, 2))
    assert bool((y == 0).all())
    dx, dg, db = torch.full_like(xv, 5.0), torch.ones(16, device="cuda"), torch.ones(16, device="cuda")
    m, r = torch.zeros((1, 2), device="cuda"), torch.ones((1, 2), device="cuda")
    xv.nan_to_num_()
    rz.map_group_norm_grad(torch.full_like(xv, float("inf")), xv, dx, 2, mean=m, rstd=r, dgamma=dg, dbeta=db,
                           drop=(1.0, 1, 2))
    assert bool((dx == 0).all()) and bool((dg == 0).all()) and bool((db == 0).all())


def test_same_bits_again_and_on_another_stream(rz):
    x = features((3, 40, 40, 64), "bf16", 10)
    a = check_forward(rz, x, 8, "bf16", "silu", 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = check_forward(rz, x, 8, "bf16", "silu", 0.1, stream=s)
    c = check_forward(rz, x, 8, "bf16", "silu", 0.1, stream=s.cuda_stream)
    assert torch.equal(a, b) and torch.equal(a, c)


def test_empty_maps(rz):
    for shape in [(0, 4, 4, 8), (2, 0, 4, 8), (2, 4, 0, 8)]:
        x = torch.empty(shape, device="cuda")
        rz.map_group_norm(x, torch.empty_like(x), 2, act=1)
        dg, db = torch.ones(8, device="cuda"), torch.ones(8, device="cuda")
        m = torch.zeros((shape[0], 2), device="cuda")
        rz.map_group_norm_grad(x, x, torch.empty_like(x), 2, mean=m, rstd=m, dgamma=dg, dbeta=db)
        assert bool((dg == 0).all()) and bool((db == 0).all())


def test_gradients_left_out(rz):
    x = features((2, 5, 5, 16), "f32", 11)
    xv, _ = ref.device_map(x, "f32")
    m, r = torch.zeros((2, 4), device="cuda"), torch.ones((2, 4), device="cuda")
    dg, db, d0, d1 = torch.empty(16, device="cuda"), torch.empty(16, device="cuda"), torch.empty_like(xv), torch.empty_like(xv)
    rz.map_group_norm_grad(xv, xv, d0, 4, mean=m, rstd=r, dgamma=dg, dbeta=db)
    rz.map_group_norm_grad(xv, xv, d1, 4, mean=m, rstd=r)
    one = torch.empty(16, device="cuda")
    rz.map_group_norm_grad(xv, xv, d1, 4, mean=m, rstd=r, dbeta=one)
    assert torch.equal(d0, d1) and torch.equal(one, db)


def test_captured_in_a_graph(rz):
    x = features((2, 16, 16, 64), "bf16", 12)
    xv, _ = ref.device_map(x, "bf16")
    y, dx = torch.empty_like(xv), torch.empty_like(xv)
    m, r = torch.empty((2, 8), device="cuda"), torch.empty((2, 8), device="cuda")
    dg, db = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    ws = torch.empty(rz.map_group_norm_workspace(xv, 8), dtype=torch.uint8, device="cuda")

    def step(s=None):
        rz.map_group_norm(xv, y, 8, mean=m, rstd=r, act=1, drop=(0.1, 4, 0), workspace=ws, stream=s)
        rz.map_group_norm_grad(y, xv, dx, 8, mean=m, rstd=r, dgamma=dg, dbeta=db, act=1, drop=(0.1, 4, 0),
                               workspace=ws, stream=s)

    step()
    want = [t.clone() for t in (y, dx, dg, db)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(torch.cuda.current_stream())
    for t in (y, dx, dg, db, ws):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dg, db)))


def test_offsets_past_32_bits(rz):
    # nine images of 2^28 elements: the last lies past 2^31 elements and 2^32 bytes
    x = torch.empty((9, 512, 512, 1024), dtype=torch.bfloat16, device="cuda")
    x.normal_()
    y, m, r = torch.empty_like(x), torch.empty((9, 32), device="cuda"), torch.empty((9, 32), device="cuda")
    rz.map_group_norm(x, y, 32, mean=m, rstd=r, act=1)
    for n in (0, 8):
        v = x[n].float().view(-1, 32, 32)
        mean, var = v.mean((0, 2)), v.var((0, 2), correction=0)
        z = torch.nn.functional.silu((v - mean[:, None]) * torch.rsqrt(var + 1e-5)[:, None]).view(512, 512, 1024)
        # the rounding of y to bf16 (8 significant bits), and float32 roundings of statistics and activation around 1e-5
        assert bool(((y[n].float() - z).abs() <= 2.0 ** -8 * z.abs() + 2e-5).all())
    dx, dg, db = torch.empty_like(x), torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    rz.map_group_norm_grad(y, x, dx, 32, mean=m, rstd=r, dgamma=dg, dbeta=db, act=0)
    n = 8
    xh = (x[n].float().view(-1, 32, 32) - m[n][:, None]) * r[n][:, None]
    d = y[n].float().view(-1, 32, 32)
    w = (d - d.mean((0, 2))[:, None] - xh * (d * xh).mean((0, 2))[:, None]) * r[n][:, None]
    w = w.view(512, 512, 1024)
    assert bool(((dx[n].float() - w).abs() <= 2.0 ** -8 * w.abs() + 2e-5).all())


def test_gradient_against_differences(rz):
    # float32 gradients against differences of the 64-bit loss: the loss's own
    # curvature term is below 1e-6 of it at this step, the float32 one below 1e-4
    x = features((2, 6, 5, 12), "f32", 13)
    gamma, beta = params(12, 14)
    dy = features(x.shape, "f32", 15)
    factor = ref.drop_factor(x.shape, 0.2, 5, 6)
    xv, _ = ref.device_map(x, "f32")
    dv, _ = ref.device_map(dy, "f32")
    y, dx = torch.empty_like(xv), torch.empty_like(xv)
    m, r = torch.empty((2, 3), device="cuda"), torch.empty((2, 3), device="cuda")
    dg, db = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
    kw = dict(act=1, eps=1e-3, drop=(0.2, 5, 6))
    rz.map_group_norm(xv, y, 3, cuda(gamma), cuda(beta), m, r, **kw)
    rz.map_group_norm_grad(dv, xv, dx, 3, cuda(gamma), cuda(beta), m, r, dg, db, **kw)
    rng, h = np.random.default_rng(16), 1e-5

    def loss(x, gamma, beta):
        return (dy * ref.group_norm(x, 3, gamma, beta, "silu", float(np.float32(1e-3)), factor)[0]).sum()

    for _ in range(4):
        vx, vg, vb = rng.normal(size=x.shape), rng.normal(size=12), rng.normal(size=12)
        slope = (loss(x + h * vx, gamma + h * vg, beta + h * vb) - loss(x - h * vx, gamma - h * vg, beta - h * vb)) / (2 * h)
        got = (ref.host(dx) * vx).sum() + (ref.host(dg) * vg).sum() + (ref.host(db) * vb).sum()
        size = np.abs(ref.host(dx) * vx).sum() + np.abs(ref.host(dg) * vg).sum()
        assert abs(got - slope) <= 1e-5 * size


def test_refusals(rz):
    x = torch.zeros((2, 4, 4, 12), device="cuda")
    y, f = torch.empty_like(x), torch.zeros(12, device="cuda")
    m = torch.zeros((2, 3), device="cuda")

    def arg(fn):
        with pytest.raises(rz.ResizeError) as e:
            fn()
        assert e.value.code == rz.RZ_ERR_ARG

    arg(lambda: rz.map_group_norm(x, y, 5))
    arg(lambda: rz.map_group_norm(x, y, 0))
    arg(lambda: rz.map_group_norm(x, y, 3, act=3))
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        arg(lambda: rz.map_group_norm(x, y, 3, eps=eps))
    for p in (-0.1, 1.1, float("nan")):
        arg(lambda: rz.map_group_norm(x, y, 3, drop=(p, 0, 0)))
    arg(lambda: rz.map_group_norm(x, x, 3))
    flat = torch.zeros(2 * 4 * 4 * 12 + 8, device="cuda")
    arg(lambda: rz.map_group_norm(flat[:384].view(2, 4, 4, 12), flat[8:].view(2, 4, 4, 12), 3))
    arg(lambda: rz.map_group_norm_grad(x, y, x, 3, mean=m, rstd=m))
    arg(lambda: rz.map_group_norm_grad(x, y, torch.empty_like(x), 3, mean=None, rstd=m))
    for bad in (x.half(), x[:, :, :3], x.cpu()):
        with pytest.raises(ValueError):
            rz.map_group_norm(x, bad, 3)
    with pytest.raises(ValueError):
        rz.map_group_norm(x.double(), y.double(), 3)
    with pytest.raises(ValueError):
        rz.map_group_norm(x.permute(0, 3, 1, 2), y.permute(0, 3, 1, 2), 2)
    with pytest.raises(ValueError):
        rz.map_group_norm(x, y, 3, gamma=f[:6])
    with pytest.raises(ValueError):
        rz.map_group_norm(x, y, 3, gamma=f.half())
    with pytest.raises(ValueError):
        rz.map_group_norm(x, y, 3, mean=torch.zeros((2, 4), device="cuda"))
