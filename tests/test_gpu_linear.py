"""Linear layer of a map with bias, activation and residual, and its gradient,
against the 64-bit forms."""
import numpy as np
import pytest

import map_reference as ref
import token_reference as tok

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ACTS = {"none": 0, "silu": 1, "gelu": 2}
TYPES = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def values(shape, dtype, seed, scale=1.0):
    return tok.rounded(np.random.default_rng(seed).normal(size=shape) * scale, dtype)


def matrix(a, dtype, pad=0, offset=0, fill=0.0):
    """A matrix with `pad` elements after each row, from element `offset` of a flat buffer."""
    rows, cols = a.shape
    flat = torch.full((offset + rows * (cols + pad) + 64,), fill, dtype=getattr(torch, tok.TORCH[dtype]), device="cuda")
    view = torch.as_strided(flat, (rows, cols), (cols + pad, 1), offset)
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(view.dtype))
    return view, flat


def check(got, want, bound, what):
    err = np.abs(ref.host(got) - want)
    assert np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-300)).max()))


def forward(rz, shape, K, dtype, kind, bias=True, residual=False, pre=False, layout={}, pad=0, offset=0, seed=1, in_place=False,
            **kw):
    C = shape[3]
    x, w = values(shape, dtype, seed), values((K, C), dtype, seed + 1, C ** -0.5)
    b = values(K, "f32", seed + 2, 0.3) if bias else None
    r = values((*shape[:3], K), dtype, seed + 3) if residual else None
    xv, _ = ref.device_map(x, dtype, **layout)
    wv, _ = matrix(w, dtype, pad, offset)
    yv, flat = ref.device_map(np.zeros((*shape[:3], K)) if not in_place else r, dtype, fill=-3.0, **layout)
    rv = None if r is None else yv if in_place else ref.device_map(r, dtype, **layout)[0]
    pv, pflat = ref.device_map(np.zeros((*shape[:3], K)), dtype, fill=-3.0, **layout) if pre else (None, None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rz.map_linear(xv, yv, wv, None if b is None else torch.from_numpy(b).float().cuda(), residual=rv, pre=pv, act=ACTS[kind],
                  status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    ty, tz = tok.linear_bounds(x, w, b, kind, r, dtype)
    want, z = tok.linear(x, w, b, kind, r)
    check(yv, want, ty, "y")
    assert ref.outside_untouched(flat, yv, -3.0)
    if pre:
        check(pv, z, tz, "pre")
        assert ref.outside_untouched(pflat, pv, -3.0)
    return yv


def gradient(rz, shape, K, dtype, kind, layout={}, pad=0, offset=0, seed=11, wdtype=None, parts="xwb", **kw):
    C = shape[3]
    wdtype = wdtype or dtype
    x, w = values(shape, dtype, seed), values((K, C), dtype, seed + 1, C ** -0.5)
    dy, pre = values((*shape[:3], K), dtype, seed + 2), values((*shape[:3], K), dtype, seed + 3, 1.5)
    xv, dv, pv = (ref.device_map(a, dtype, **layout)[0] for a in (x, dy, pre))
    wv, _ = matrix(w, dtype, pad, offset)
    ov, oflat = ref.device_map(np.zeros(shape), dtype, fill=-3.0, **layout)
    gv, gflat = matrix(np.zeros((K, C)), wdtype, pad, offset, -3.0)
    gv.fill_(7.0)
    db = torch.full((K,), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rz.map_linear_grad(dv, xv, wv, ov if "x" in parts else None, gv if "w" in parts else None, db if "b" in parts else None,
                       pre=None if kind == "none" else pv, act=ACTS[kind], status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    dx, dw, dbias, _ = tok.linear_grad(dy, x, w, pre, kind)
    tx, tw, tb = tok.linear_grad_bounds(dy, x, w, pre, kind, dtype, wdtype)
    if "x" in parts:
        check(ov, dx, tx, "dx")
    if "w" in parts:
        check(gv, dw, tw, "dweight")
    if "b" in parts:
        check(db, dbias, tb, "dbias")
    assert ref.outside_untouched(oflat, ov, -3.0) and ref.outside_untouched(gflat, gv, -3.0)
    return ov, gv, db


# (N, H, W, C), K: one value; one pixel; widths of one; widths that fill no vector, no tile; tiles just filled and just passed
SHAPES = [((1, 1, 1, 1), 1), ((1, 1, 1, 640), 96), ((1, 1, 1, 37), 5), ((2, 1, 1, 256), 130), ((7, 1, 1, 512), 64),
          ((9, 1, 1, 72), 1000), ((2, 3, 5, 1), 7), ((2, 3, 5, 9), 1), ((1, 8, 16, 64), 64), ((1, 9, 15, 65), 63),
          ((3, 13, 11, 96), 250), ((2, 16, 16, 128), 256), ((1, 17, 31, 200), 322), ((1, 1, 130, 264), 520),
          ((1, 40, 33, 16), 24), ((1, 1, 300, 1030), 8)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape, K", SHAPES)
def test_forward(rz, shape, K, dtype):
    forward(rz, shape, K, dtype, "gelu", residual=True, pre=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape, K", SHAPES)
def test_gradient(rz, shape, K, dtype):
    gradient(rz, shape, K, dtype, "silu")


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("bias, residual, pre", [(True, False, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((3, 1, 1, 72), 136), ((2, 9, 15, 21), 33)])
def test_epilogues(rz, kind, bias, residual, pre, dtype, shape, K):
    forward(rz, shape, K, dtype, kind, bias, residual, pre)


@pytest.mark.parametrize("kind", list(ACTS))
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((3, 1, 1, 72), 136), ((2, 9, 15, 21), 33)])
def test_slopes(rz, kind, dtype, shape, K):
    gradient(rz, shape, K, dtype, kind)


@pytest.mark.parametrize("parts", ["x", "w", "b", "xw", "wb", "xb"])
@pytest.mark.parametrize("kind", ["none", "gelu"])
def test_parts_of_the_gradient(rz, parts, kind):
    gradient(rz, (2, 9, 15, 72), 136, "bf16", kind, parts=parts)


# padded rows, gaps between images, starts that no vector is aligned to
LAYOUTS = [dict(pad=16), dict(gap=64), dict(pad=8, gap=24), dict(offset=1), dict(pad=4, offset=4), dict(pad=1)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [64, 50])
def test_layouts(rz, layout, dtype, K):
    forward(rz, (2, 11, 13, 32), K, dtype, "silu", residual=True, pre=True, layout=layout)
    gradient(rz, (2, 11, 13, 32), K, dtype, "gelu", layout)


@pytest.mark.parametrize("pad, offset", [(8, 0), (0, 1), (3, 2), (8, 8)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(2, 11, 13, 40), (1, 1, 2, 40)])
def test_weights_with_padding(rz, pad, offset, dtype, shape):
    forward(rz, shape, 56, dtype, "none", pad=pad, offset=offset)
    gradient(rz, shape, 56, dtype, "none", pad=pad, offset=offset)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["none", "silu"])
def test_weight_gradient_in_float32(rz, dtype, kind):
    gradient(rz, (2, 9, 15, 72), 136, dtype, kind, wdtype="f32")


@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((4, 1, 1, 72), 136)])
@pytest.mark.parametrize("dtype", TYPES)
def test_residual_in_place(rz, shape, K, dtype):
    forward(rz, shape, K, dtype, "none", residual=True, in_place=True)


# sums over many pixels, many terms, and more tiles than there are processors
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape, K", [((1, 64, 160, 24), 40), ((1, 5, 50, 4096), 72), ((2, 96, 100, 136), 328), ((2, 64, 65, 520), 520),
                                      ((1, 60, 70, 1030), 264), ((1, 40, 50, 640), 1000), ((1, 50, 60, 512), 512),
                                      ((1, 30, 40, 1024), 1024)])
def test_larger(rz, shape, K, dtype):
    forward(rz, shape, K, dtype, "silu", residual=True, pre=True)
    gradient(rz, shape, K, dtype, "gelu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((1, 40, 50, 200), 72), ((3, 1, 1, 512), 136)])
def test_same_bits_every_time(rz, shape, K, dtype):
    a = forward(rz, shape, K, dtype, "gelu").clone()
    g = [t.clone() for t in gradient(rz, shape, K, dtype, "gelu")]
    for _ in range(3):
        assert torch.equal(a, forward(rz, shape, K, dtype, "gelu"))
        assert all(torch.equal(u, v) for u, v in zip(g, gradient(rz, shape, K, dtype, "gelu")))


@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((1, 40, 50, 200), 72), ((3, 1, 1, 512), 136)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_other_stream_and_given_workspace(rz, shape, K, dtype):
    x = torch.zeros(shape, dtype=getattr(torch, tok.TORCH[dtype]), device="cuda")
    y = torch.zeros((*shape[:3], K), dtype=x.dtype, device="cuda")
    w = torch.zeros((K, shape[3]), dtype=x.dtype, device="cuda")
    n = max(rz.map_linear_workspace(x, y, w, act=1), rz.map_linear_grad_workspace(y, x, w, x, w, pre=y, act=1))
    work = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        forward(rz, shape, K, dtype, "silu", workspace=work[:n], stream=s)
        gradient(rz, shape, K, dtype, "silu", workspace=work[:n], stream=s)
    assert bool((work[n:] == 0xA5).all())


@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((1, 40, 50, 200), 72), ((3, 1, 1, 512), 136)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(rz, shape, K, dtype):
    C = shape[3]
    t = getattr(torch, tok.TORCH[dtype])
    x, dy, pre = (torch.zeros(s, dtype=t, device="cuda") for s in (shape, (*shape[:3], K), (*shape[:3], K)))
    w, y, dx = torch.zeros((K, C), dtype=t, device="cuda"), torch.zeros_like(dy), torch.zeros_like(x)
    dw, db = torch.zeros_like(w), torch.zeros(K, device="cuda")
    fw = torch.empty(max(16, rz.map_linear_workspace(x, y, w, pre=pre, act=2)), dtype=torch.uint8, device="cuda")
    gw = torch.empty(max(16, rz.map_linear_grad_workspace(dy, x, w, dx, dw, pre, act=2)), dtype=torch.uint8, device="cuda")

    def step():
        rz.map_linear(x, y, w, pre=pre, act=2, workspace=fw)
        rz.map_linear_grad(dy, x, w, dx, dw, db, pre=pre, act=2, workspace=gw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        vx, vw, vd = values(shape, dtype, seed), values((K, C), dtype, seed + 5, C ** -0.5), values((*shape[:3], K), dtype, seed + 7)
        for a, v in ((x, vx), (w, vw), (dy, vd)):
            a.copy_(torch.from_numpy(v).to(t))
        g.replay()
        torch.cuda.synchronize()
        check(y, tok.linear(vx, vw, None, "gelu")[0], tok.linear_bounds(vx, vw, None, "gelu", None, dtype)[0], "y")
        p = ref.host(pre)
        want = tok.linear_grad(vd, vx, vw, p, "gelu")
        for a, v, b, name in zip((dx, dw, db), want, tok.linear_grad_bounds(vd, vx, vw, p, "gelu", dtype, dtype), ("dx", "dw", "db")):
            check(a, v, b, name)


@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_in_their_rows(rz, dtype):
    shape, K = (1, 9, 17, 72), 136
    x, w = values(shape, dtype, 3), values((K, 72), dtype, 4, 0.1)
    xv, wv = (torch.from_numpy(a).to(getattr(torch, tok.TORCH[dtype])).cuda() for a in (x, w))
    xv[0, 2, 3, 7] = float("nan")
    xv[0, 5, 1, 0] = float("inf")
    y = torch.empty((1, 9, 17, K), dtype=xv.dtype, device="cuda")
    rz.map_linear(xv, y, wv)
    bad = torch.zeros((1, 9, 17), dtype=torch.bool)
    bad[0, 2, 3] = bad[0, 5, 1] = True
    assert not bool(torch.isfinite(y.cpu()[bad]).any())
    assert bool(torch.isfinite(y.cpu()[~bad]).all())


def test_empty_maps(rz):
    for shape in ((0, 3, 3, 16), (2, 0, 3, 16), (2, 3, 0, 16)):
        x, y = torch.empty(shape, device="cuda"), torch.empty((*shape[:3], 24), device="cuda")
        w, dw, db = torch.ones((24, 16), device="cuda"), torch.full((24, 16), 5.0, device="cuda"), torch.full((24,), 5.0, device="cuda")
        rz.map_linear(x, y, w)
        rz.map_linear_grad(y, x, w, torch.empty_like(x), dw, db)
        assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0


@pytest.mark.parametrize("kind", list(ACTS))
def test_gradient_against_differences(rz, kind):
    """d(sum of dy y) along random directions, by central differences of the float32 forward, in float64."""
    shape, K, h = (2, 5, 7, 24), 40, 2.0 ** -6
    x, w, b, dy = (values(s, "f32", i) for i, s in enumerate((shape, (K, 24), (K,), (*shape[:3], K))))
    gpu = lambda a: torch.from_numpy(a).float().cuda()    # noqa: E731
    y, pre = torch.empty((*shape[:3], K), device="cuda"), torch.empty((*shape[:3], K), device="cuda")
    dx, dw, db = torch.empty(shape, device="cuda"), torch.empty((K, 24), device="cuda"), torch.empty(K, device="cuda")
    rz.map_linear(gpu(x), y, gpu(w), gpu(b), pre=pre, act=ACTS[kind])
    rz.map_linear_grad(gpu(dy), gpu(x), gpu(w), dx, dw, db, pre=pre, act=ACTS[kind])
    rng = np.random.default_rng(7)
    for k, (v, g) in enumerate(((x, dx), (w, dw), (b, db))):
        d = rng.normal(size=v.shape)
        d /= np.linalg.norm(d)
        sums = []
        for s in (1, -1):
            a = [x, w, b]
            a[k] = tok.rounded(v + s * h * d, "f32")
            rz.map_linear(gpu(a[0]), y, gpu(a[1]), gpu(a[2]), act=ACTS[kind])
            sums.append(float((ref.host(y) * dy).sum()))
        slope = (sums[0] - sums[1]) / (2 * h)
        # float32 forwards: 88 U of each |y| before the division by 2 h, random over the sum's n terms (six deviations); the
        # third derivative's h^2 / 6 of a smooth sum: 1e-3 of its size
        noise = 6 * 88 * 2.0 ** -24 * np.linalg.norm(ref.host(y) * dy) / h + 1e-3 * np.linalg.norm(ref.host(g))
        assert abs(slope - float((ref.host(g) * d).sum())) <= noise


def test_calls_without_a_status_word_report_to_the_bindings_own(rz):
    x, w = torch.ones((1, 4, 8, 16), device="cuda"), torch.ones((24, 16), device="cuda")
    y, dw = torch.empty((1, 4, 8, 24), device="cuda"), torch.empty((24, 16), device="cuda")
    rz.map_linear(x, y, w)
    word, at, kept = rz._waits[0]
    assert at == kept.data_ptr() and kept.is_pinned() and word.value == 0
    # the device can write it where the host reads it
    device_view = torch.tensor([7], dtype=torch.int32, device="cuda")
    kept.copy_(device_view)
    torch.cuda.synchronize()
    with pytest.raises(rz.ResizeError, match="earlier"):
        rz.map_linear_grad(y, x, w, None, dw)
    rz.map_linear_grad(y, x, w, None, dw)
    torch.cuda.synchronize()
    assert word.value == 0 and float(dw[0, 0]) == 32 * 16
    s = torch.cuda.Stream()
    assert not rz._capturing(None) and not rz._capturing(s) and not rz._capturing(s.cuda_stream)
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        assert rz._capturing(None) and rz._capturing(s)
        rz.map_linear(x, y, w)


def test_first_call_inside_a_capture(rz, monkeypatch):
    monkeypatch.setattr(rz, "_waits", {})
    x, w, y = (torch.ones(s, device="cuda") for s in ((1, 4, 8, 16), (24, 16), (1, 4, 8, 24)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rz.map_linear(x, y, w)
    assert not rz._waits
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert bool((y == 16).all())


def gelu_border(dtype, k):
    """Float32 z whose GELU lies (k + 3 |z|) |z| / 2^26 or just more from where its rounding changes, on either side, and what
    it rounds to: an error of that size turns the rounding."""
    import scipy.special as sp

    def f(z):
        return z * sp.ndtr(z)

    t = getattr(torch, tok.TORCH[dtype])
    rng = np.random.default_rng(9)
    found = []
    # an interval of z, whether GELU rises there, and borders: the middles of neighbours of the type
    for lo, hi, rises in ((2.0 ** -9, 7.0, True), (-0.7, -(2.0 ** -9), True), (-3.0, -0.8, False)):
        one = np.sign(lo) * 2.0 ** rng.uniform(*np.sort(np.log2(np.abs([lo, hi]))), 12000)
        g = torch.unique(torch.from_numpy(f(one)).to(t))
        border = ((g.double() + (g.view(torch.int16) + 1).view(t).double()) / 2).numpy()
        for side in (-1, 1):
            a, b = np.full(border.shape, lo), np.full(border.shape, hi)
            for _ in range(200):
                m = (a + b) / 2
                above = f(m) - side * (k + 3 * np.abs(m)) * np.abs(m) / 2 ** 26 > border
                up = above == rises
                a, b = np.where(up, a, m), np.where(up, m, b)
            z = ((a + b) / 2).astype(np.float32)
            # the next float32 on the far side of the margin
            for _ in range(4):
                z64 = z.astype(np.float64)
                margin = side * (f(z64) - border) - (k + 3 * np.abs(z64)) * np.abs(z64) / 2 ** 26
                away = np.float32(np.inf if (side > 0) == rises else -np.inf)
                z = np.where(margin < 0, np.nextafter(z, away), z)
            z64 = z.astype(np.float64)
            margin = side * (f(z64) - border) - (k + 3 * np.abs(z64)) * np.abs(z64) / 2 ** 26
            good = (margin >= 0) & (margin < 4 * np.abs(z64) / 2 ** 24) & (z64 > lo) & (z64 < hi)
            found.append(z64[good])
    z = np.unique(np.concatenate(found))
    return z, torch.from_numpy(f(z)).to(t).double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pixels", [1, 40])
def test_gelu_of_16_bit_maps_is_as_good_as_stated(rz, dtype, pixels):
    """(25 + 3 |z|) |z| / 2^26 before the rounding: z by way of the bias."""
    z, want = gelu_border(dtype, 25)
    assert z.size > (200 if dtype == "bf16" else 4000)
    t = getattr(torch, tok.TORCH[dtype])
    y = torch.empty((1, 1, pixels, z.size), dtype=t, device="cuda")
    rz.map_linear(torch.zeros((1, 1, pixels, 8), dtype=t, device="cuda"), y, torch.zeros((z.size, 8), dtype=t, device="cuda"),
                  torch.from_numpy(z).float().cuda(), act=ACTS["gelu"])
    assert np.array_equal(ref.host(y), np.broadcast_to(want, y.shape))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gelu_of_16_bit_maps_far_below_zero(rz, dtype):
    """3e-4 of the tail before the rounding."""
    import scipy.special as sp
    z = -np.linspace(2.0, 5.9, 60000).astype(np.float32).astype(np.float64)
    t = getattr(torch, tok.TORCH[dtype])
    y = torch.empty((1, 1, 1, z.size), dtype=t, device="cuda")
    rz.map_linear(torch.zeros((1, 1, 1, 8), dtype=t, device="cuda"), y, torch.zeros((z.size, 8), dtype=t, device="cuda"),
                  torch.from_numpy(z).float().cuda(), act=ACTS["gelu"])
    want = z * sp.ndtr(z)
    check(y, want, ref.stored(want, 3e-4 * np.abs(want), dtype), "y")


# The error of a float32 result of n terms, of the sum S of their magnitudes.  The tensor cores cut what they add: a run of
# r terms of one sign and alike in size ends up short by 3e-9 r at most (float16 operands: 8e-9 r, their products have more
# bits), the same way every time, runs being 512 terms of float32 operands and 1024 of 16-bit ones at most.  The products of
# planes that are left out hold 2^-21 of a term at most.  Runs are added in float32, each rounding 2^-24 at most of what is
# there, of random sign: six deviations of as many as there are runs.
def held(n, dtype):
    run = 512 if dtype == "f32" else 1024
    cut = min(n, run) * (8e-9 if dtype == "f16" else 3e-9)
    return cut + (2.0 ** -21 if dtype == "f32" else 0.0) + 6 * np.sqrt(np.ceil(n / run)) * 2.0 ** -24


def near(got, a, b, bound):
    """got against a @ b in float64, off by at most `bound` of the magnitudes' sums."""
    want, S = a.double() @ b.double(), a.double().abs() @ b.double().abs()
    return float(((got.double() - want).abs() / S).max()) <= bound


@pytest.mark.parametrize("positive", [True, False])
@pytest.mark.parametrize("P, C, K", [(300, 200, 64), (300, 1024, 72), (130, 4096, 40), (100, 65536, 8), (5000, 1536, 1000)])
def test_float32_products_are_as_good_as_stated(rz, positive, P, C, K):
    """All terms positive: what is cut adds up, and nothing hides in a cancelled sum."""
    g = torch.Generator(device="cuda").manual_seed(C)
    x, w = (torch.rand(s, generator=g, device="cuda") - (0.0 if positive else 0.5) for s in ((1, 1, P, C), (K, C)))
    y = torch.empty((1, 1, P, K), device="cuda")
    rz.map_linear(x, y, w)
    assert near(y[0, 0], x[0, 0], w.T, held(C, "f32"))
    dy = torch.rand((1, 1, P, K), generator=g, device="cuda") - (0.0 if positive else 0.5)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    rz.map_linear_grad(dy, x, w, dx, dw)
    assert near(dx[0, 0], dy[0, 0], w, held(K, "f32"))
    assert near(dw, dy[0, 0].T, x[0, 0], held(P, "f32"))


@pytest.mark.parametrize("positive", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P, C, K", [(65536, 64, 64), (65536, 40, 264), (20000, 256, 512), (200000, 8, 16)])
def test_float32_weight_gradients_are_as_good_as_stated(rz, positive, dtype, P, C, K):
    g = torch.Generator(device="cuda").manual_seed(P + C)
    t = getattr(torch, tok.TORCH[dtype])
    x, dy = ((torch.rand((1, 1, P, n), generator=g, device="cuda") - (0.0 if positive else 0.5)).to(t) for n in (C, K))
    dw, db = torch.empty((K, C), device="cuda"), torch.empty(K, device="cuda")
    rz.map_linear_grad(dy, x, torch.zeros((K, C), dtype=t, device="cuda"), None, dw, db)
    assert near(dw, dy[0, 0].T, x[0, 0], held(P, dtype))
    assert near(db[:, None], dy[0, 0].T, torch.ones((P, 1), device="cuda"), tok.walk(min(P, 4096)) * 2.0 ** -24)
    again = torch.empty_like(dw)
    rz.map_linear_grad(dy, x, torch.zeros((K, C), dtype=t, device="cuda"), None, again)
    assert torch.equal(dw, again)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype, left", [("bf16", 2.0 ** -16), ("f16", 2.0 ** -22)])
@pytest.mark.parametrize("shape, K", [((2, 9, 15, 72), 136), ((1, 40, 50, 64), 128), ((1, 30, 70, 37), 51), ((1, 1, 5, 16), 24)])
def test_float32_weight_gradients_see_dz_whole(rz, kind, dtype, left, shape, K):
    """dz as the sum of two values of the type: half a step of the second is left of it (`left` of dz, and half a step of
    float16's smallest), where a 16-bit dweight sees half a step of the first."""
    C, P = shape[3], shape[0] * shape[1] * shape[2]
    x, dy, pre = values(shape, dtype, 1), values((*shape[:3], K), dtype, 2), values((*shape[:3], K), dtype, 3, 1.5)
    x, dy = np.abs(x), np.abs(dy)           # of one sign, so that nothing cancels
    t = getattr(torch, tok.TORCH[dtype])
    xv, dv, pv = (torch.from_numpy(a).to(t).cuda() for a in (x, dy, pre))
    dx, dw, db = torch.empty_like(xv), torch.empty((K, C), device="cuda"), torch.empty(K, device="cuda")
    w = values((K, C), dtype, 4, C ** -0.5)
    wv = torch.from_numpy(w).to(t).cuda()
    rz.map_linear_grad(dv, xv, wv, dx, dw, db, pre=pv, act=ACTS[kind])
    want = tok.linear_grad(dy, x, w, pre, kind)
    dz, xa = np.abs(want[3]).reshape(P, K), x.reshape(P, C)
    slope = (dy * ref.slope_error(pre, 0, kind)).reshape(P, K) + 2.0 ** -24 * dz
    bound = (slope + left * dz + (2.0 ** -25 if dtype == "f16" else 0.0)).T @ xa + held(P, dtype) * (dz.T @ xa)
    check(dw, want[1], bound, "dweight")
    # the same dx and dbias as beside a dweight of the type
    other = [torch.empty_like(a) for a in (dx, wv, db)]
    rz.map_linear_grad(dv, xv, wv, *other, pre=pv, act=ACTS[kind])
    assert torch.equal(dx, other[0]) and torch.equal(db, other[2])


@pytest.mark.parametrize("act", [1, 2])
def test_float16_dz_past_its_range(rz, act):
    """An infinite first value leaves no second one: the sum stays infinite."""
    t = torch.float16
    x, w = torch.ones((1, 1, 4, 8), dtype=t, device="cuda"), torch.ones((8, 8), dtype=t, device="cuda")
    dy, pre = torch.ones((1, 1, 4, 8), dtype=t, device="cuda"), torch.full((1, 1, 4, 8), 2.0, dtype=t, device="cuda")
    dy[0, 0, 1, 3] = 65000.0                                  # times a slope of 1.09
    dw = torch.empty((8, 8), device="cuda")
    rz.map_linear_grad(dy, x, w, None, dw, pre=pre, act=act)
    assert bool(torch.isposinf(dw[3]).all()) and bool(torch.isfinite(dw[[0, 1, 2, 4, 5, 6, 7]]).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 3, 72), (1, 9, 17, 72)])
def test_infinities_keep_their_sign(rz, dtype, shape):
    """Of one infinity in a row the sums are infinite, of the sign of its product, however many rows there are; a zero's
    product is NaN."""
    K, P = 136, shape[1] * shape[2]
    t = getattr(torch, tok.TORCH[dtype])
    x, w = (torch.from_numpy(values(s, dtype, i)).to(t).cuda() for i, s in enumerate((shape, (K, 72))))
    w[::3] = torch.sign(w[::3]) * 0.5                         # values whose lower bits are 0
    w[5, 7] = 0.0
    x[0, 0, 1, 7], x[0, 0, 2, 70] = float("inf"), -float("inf")
    y = torch.empty((*shape[:3], K), dtype=t, device="cuda")
    rz.map_linear(x, y, w)
    want = x[0].double().cpu().view(P, 72) @ w.double().cpu().T
    got = y.double().cpu().view(P, K)
    assert bool(torch.isnan(want[1, 5])) and int(torch.isinf(want).sum()) == 2 * K - 1
    finite = torch.isfinite(want)
    assert torch.equal(torch.nan_to_num(got[~finite], nan=7.0), torch.nan_to_num(want[~finite], nan=7.0))
    assert bool(torch.isfinite(got[finite]).all())
    # backward: dy's infinity reaches its row of dx and its row of dweight alone
    dy = torch.from_numpy(values((*shape[:3], K), dtype, 3)).to(t).cuda()
    dy[0, 0, 2, 9] = -float("inf")
    xb = torch.from_numpy(values(shape, dtype, 4)).to(t).cuda()
    dx, dw, db = torch.empty_like(xb), torch.empty_like(w), torch.empty(K, device="cuda")
    rz.map_linear_grad(dy, xb, w, dx, dw, db)
    flat = dy.double().cpu().view(P, K)
    for got, want in ((dx.view(P, 72), flat @ w.double().cpu()), (dw, flat.T @ xb.double().cpu().view(P, 72))):
        got, odd = got.double().cpu(), ~torch.isfinite(want)
        assert torch.equal(torch.nan_to_num(got[odd], nan=7.0), torch.nan_to_num(want[odd], nan=7.0)) and bool(torch.isfinite(got[~odd]).all())
    assert float(db[9]) == -float("inf")


@pytest.mark.parametrize("pitch", [0, 2, 16, 1 << 12])
@pytest.mark.parametrize("pixels", [5, 300])
def test_weights_of_one_row_have_any_pitch(rz, pixels, pitch):
    """By the C entry: the pitch of a single row leads nowhere."""
    import ctypes

    from bilinear_image_resize_gb300 import _native
    lib, C = _native.load(), 64
    x, dy = (torch.from_numpy(values((1, 1, pixels, n), "bf16", n)).bfloat16().cuda() for n in (C, 1))
    w, y, dx = torch.from_numpy(values((1, C), "bf16", 3)).bfloat16().cuda(), torch.empty_like(dy), torch.empty_like(x)
    dw, db = torch.full((1, C), 5.0, dtype=torch.bfloat16, device="cuda"), torch.empty(1, device="cuda")
    d = _native.RzLinear(1, 1, pixels, C, 1, 2, 0)
    m = lambda t: _native.RzMap(t.data_ptr(), pixels * t.shape[3] * 2, pixels * t.shape[3] * 2)      # noqa: E731
    work = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    n = ctypes.c_size_t(0)
    assert lib.map_linear_workspace(d, m(x), w.data_ptr(), pitch, None, None, m(y), ctypes.byref(n)) == 0 and n.value <= 1 << 24
    assert lib.map_linear(d, m(x), w.data_ptr(), pitch, None, None, None, m(y), work.data_ptr(), 1 << 24, None, s) == 0
    assert lib.map_linear_grad(d, m(dy), m(x), w.data_ptr(), pitch, None, m(dx), dw.data_ptr(), pitch, 2, db.data_ptr(), work.data_ptr(),
                               1 << 24, None, s) == 0
    torch.cuda.synchronize()
    xa, wa, da = ref.host(x), ref.host(w), ref.host(dy)
    check(y, tok.linear(xa, wa, None, "none")[0], tok.linear_bounds(xa, wa, None, "none", None, "bf16")[0], "y")
    for got, want, bound in zip((dx, dw, db), tok.linear_grad(da, xa, wa, None, "none"),
                                tok.linear_grad_bounds(da, xa, wa, None, "none", "bf16", "bf16")):
        check(got, want, bound, "gradient")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C, K, P", [(37, 40, 300), (321, 136, 400), (1, 64, 300), (63, 130, 513), (45, 1, 3000), (37, 40, 5)])
def test_odd_weights_beside_values_that_are_not_finite(rz, dtype, C, K, P):
    """Rows of odd widths, 16 bytes and more apart, read where they lie: nothing of what is between them is."""
    x, w, dy = values((1, 1, P, C), dtype, 1), values((K, C), dtype, 2, C ** -0.5), values((1, 1, P, K), dtype, 3)
    t = getattr(torch, tok.TORCH[dtype])
    pad = (C + 7) // 8 * 8 + 8 - C
    wv, _ = matrix(w, dtype, pad, 0, float("nan"))
    xv, dv = (torch.from_numpy(a).to(t).cuda() for a in (x, dy))
    y, dx, db = torch.empty_like(dv), torch.empty_like(xv), torch.empty(K, device="cuda")
    gv, gflat = matrix(np.zeros((K, C)), dtype, pad, 0, -3.0)
    rz.map_linear(xv, y, wv)
    rz.map_linear_grad(dv, xv, wv, dx, gv, db)
    check(y, tok.linear(x, w, None, "none")[0], tok.linear_bounds(x, w, None, "none", None, dtype)[0], "y")
    for got, want, bound in zip((dx, gv, db), tok.linear_grad(dy, x, w, None, "none"),
                                tok.linear_grad_bounds(dy, x, w, None, "none", dtype, dtype)):
        check(got, want, bound, "gradient")
    assert ref.outside_untouched(gflat, gv, -3.0)


def test_first_call_on_a_given_stream(rz, monkeypatch):
    """The binding's status word is made on any stream, the default's number among them."""
    x, w = torch.ones((1, 4, 8, 16), device="cuda"), torch.ones((24, 16), device="cuda")
    for stream in (0, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        monkeypatch.setattr(rz, "_waits", {})
        y = torch.empty((1, 4, 8, 24), device="cuda")
        torch.cuda.synchronize()
        rz.map_linear(x, y, w, stream=stream)
        torch.cuda.synchronize()
        assert 0 in rz._waits and bool((y == 16).all())
