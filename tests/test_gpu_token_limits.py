"""The operators around attention at the ends of their ranges: images and rows that
lie past 32 bits, results of more than 4 GB, two calls at once, values at the ends
of a type's range."""
import numpy as np
import pytest

import map_reference as ref
import token_reference as tok

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

FAR = 1_200_000_008         # elements between images: two bytes each, the third image begins past 2^32 bytes


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    yield m
    torch.cuda.empty_cache()


def values(shape, dtype, seed, scale=1.0):
    return tok.rounded(np.random.default_rng(seed).normal(size=shape) * scale, dtype)


def cuda(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, tok.TORCH[dtype])).cuda()


def far(a, stride=FAR):
    """A bfloat16 copy of the array whose first axis steps by `stride` elements."""
    rest = int(np.prod(a.shape[1:]))
    flat = torch.empty((a.shape[0] - 1) * stride + rest, dtype=torch.bfloat16, device="cuda")
    inner = torch.empty(a.shape[1:], device="meta").stride()
    view = torch.as_strided(flat, a.shape, (stride, *inner))
    view.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(torch.bfloat16))
    return view


def check(got, want, bound, what):
    err = np.abs(ref.host(got) - want)
    assert np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-300)).max()))


@pytest.mark.parametrize("shape", [(3, 5, 7, 72), (3, 1, 2, 72)])
def test_linear_of_images_far_apart(rz, shape):
    K = 136
    x, w, r = values(shape, "bf16", 1), values((K, 72), "bf16", 2, 0.1), values((*shape[:3], K), "bf16", 3)
    xv, yv, wv = far(x), far(np.zeros(r.shape)), cuda(w, "bf16")
    rv = far(r)
    rz.map_linear(xv, yv, wv, residual=rv, act=1)
    check(yv, tok.linear(x, w, None, "silu", r)[0], tok.linear_bounds(x, w, None, "silu", r, "bf16")[0], "y")
    ov, gv, db = far(np.zeros(shape)), torch.empty_like(wv), torch.empty(K, device="cuda")
    rz.map_linear_grad(rv, xv, wv, ov, gv, db)
    want = tok.linear_grad(r, x, w, None, "none")
    for a, v, b, name in zip((ov, gv, db), want, tok.linear_grad_bounds(r, x, w, None, "none", "bf16", "bf16"), ("dx", "dw", "db")):
        check(a, v, b, name)


@pytest.mark.parametrize("pixels", [2, 300])
def test_linear_of_weight_rows_far_apart(rz, pixels):
    shape, K = (1, 1, pixels, 64), 80
    x, w, d = values(shape, "bf16", 1), values((K, 64), "bf16", 2, 0.1), values((1, 1, pixels, K), "bf16", 3)
    wv, gv = far(w, (1 << 25) + 8), far(np.zeros((K, 64)), (1 << 25) + 16)
    xv, y = cuda(x, "bf16"), torch.empty((1, 1, pixels, K), dtype=torch.bfloat16, device="cuda")
    rz.map_linear(xv, y, wv)
    check(y, tok.linear(x, w, None, "none")[0], tok.linear_bounds(x, w, None, "none", None, "bf16")[0], "y")
    dx = torch.empty_like(xv)
    rz.map_linear_grad(cuda(d, "bf16"), xv, wv, dx, gv)
    want, bounds = tok.linear_grad(d, x, w, None, "none"), tok.linear_grad_bounds(d, x, w, None, "none", "bf16", "bf16")
    check(dx, want[0], bounds[0], "dx")
    check(gv, want[1], bounds[1], "dweight")


def test_linear_of_more_than_four_gigabytes(rz):
    P, C, K = 2_200_000, 64, 1024
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((1, 1100, 2000, C), generator=g, device="cuda").bfloat16()
    w = (torch.randn((K, C), generator=g, device="cuda") / 8).bfloat16()
    y = torch.empty((1, 1100, 2000, K), dtype=torch.bfloat16, device="cuda")
    rz.map_linear(x, y, w)
    flat, rows = x.view(P, C), y.view(P, K)
    u = 2.0 ** -8

    def near(got, a, b):
        want, S = a @ b, a.abs() @ b.abs()
        # a float32 sum, rounded once
        e = tok.sum_error(a.shape[1], S)
        return bool(((got.double() - want).abs() <= e * (1 + u) + u * want.abs()).all())

    for at in (0, 999, 1 << 20, (1 << 21) - 64, (1 << 21) + 3, P - 64):        # 2^21 rows are 2^32 bytes
        assert near(rows[at:at + 64], flat[at:at + 64].double(), w.double().T)
    dx, dw = torch.empty_like(x), torch.empty((K, C), device="cuda")
    rz.map_linear_grad(y, x, w, dx, dw)
    for at in (0, 1 << 20, (1 << 21) - 64, P - 64):
        assert near(dx.view(P, C)[at:at + 64], rows[at:at + 64].double(), w.double())
    want, S = torch.zeros((K, C), dtype=torch.float64, device="cuda"), torch.zeros((K, C), dtype=torch.float64, device="cuda")
    for p in range(0, P, 100_000):
        a, b = rows[p:p + 100_000].double().T, flat[p:p + 100_000].double()
        want += a @ b
        S += a.abs() @ b.abs()
    # a run's sum on the tensor cores is cut once for 16 of its 2048 terms, 2 U each; the runs, about P / 2048, are added in order
    e = (2 * 2048 / 16 + P / 2048 + 64) * 2.0 ** -24 * S
    assert bool(((dw.double() - want).abs() <= e).all())


def test_qk_norm_of_images_far_apart(rz):
    grid, D = (3, 3, 5), 32
    x, dy = values((*grid, 96), "bf16", 1), values((*grid, 64), "bf16", 2)
    xv, yv, dv, ov = far(x), far(np.zeros(dy.shape)), far(dy), far(np.zeros(x.shape))
    one, t, eps = np.ones(D), tok.angles(*grid, D, None, 100.0, 8, 8, 1.0), float(np.float32(1e-6))
    turn = dict(base=100.0, row_pairs=8, col_pairs=8)
    rz.map_qk_norm(xv, yv, 1, 1, D, **turn)
    want, err = tok.qk_norm(x, 1, 1, D, one, one, t, False, eps)
    check(yv, want, ref.stored(want, err, "bf16"), "y")
    rz.map_qk_norm_grad(dv, xv, ov, 1, 1, D, **turn)
    dx, _, _, ex, _, _ = tok.qk_norm_grad(dy, x, 1, 1, D, one, one, t, False, eps)
    check(ov[..., :64], dx, ref.stored(dx, ex, "bf16"), "dx")


@pytest.mark.parametrize("rows_apart", [False, True])
@pytest.mark.parametrize("N", [1, 9, 40])
def test_position_bias_of_matrices_far_apart(rz, N, rows_apart):
    query, key, heads, R = (5, 8), (5, 8), 3, 11
    rule = (4, 6, 20)
    rows, cols = tok.buckets(5, 5, *rule), tok.buckets(8, 8, *rule)
    table, s = values((R, R, heads), "f32", 1), values((N, heads, 40, 40), "bf16", 2)
    if rows_apart:
        step = 2_400_000_016 // (N * heads * 40) // 8 * 8
        stride = 40 * step
    else:
        step, stride = 40, 3_000_000_008 // (N * heads) // 8 * 8

    def spread(a):
        flat = torch.empty((N * heads - 1) * stride + 39 * step + 40, dtype=torch.bfloat16, device="cuda")
        view = torch.as_strided(flat, a.shape, (heads * stride, stride, step, 1))
        view.copy_(cuda(a, "bf16"))
        return view

    t, r, c = cuda(table), torch.from_numpy(rows).int().cuda(), torch.from_numpy(cols).int().cuda()
    sv, out = spread(s), spread(np.zeros(s.shape))
    rz.map_position_bias(t, r, c, out, query, key, scores=sv)
    want = s + tok.position_bias(table, rows, cols, query, key)
    assert np.all(np.abs(ref.host(out) - want) <= ref.stored(want, 2.0 ** -24 * np.abs(want), "bf16"))
    dt = torch.empty((R, R, heads), device="cuda")
    rz.map_position_bias_grad(sv, r, c, dt, query, key)
    w, mag, count = tok.position_bias_grad(s, rows, cols, query, key, R, R)
    steps = np.vectorize(ref.walk)(np.maximum(count, 1))[..., None]
    assert np.all(np.abs(ref.host(dt) - w) <= 2.0 ** -24 * (steps * mag + np.abs(w)))


def test_two_calls_at_once(rz):
    """Calls on two streams, in turn, give what each gives alone."""
    def inputs(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
        return dict(x=new(2, 48, 50, 512), w=new(1024, 512) / 16, dy=new(2, 48, 50, 1024), q=new(2, 48, 50, 384), s=new(2, 4, 400, 400),
                    t=torch.randn((39, 39, 4), generator=g, device="cuda"))

    lut = torch.arange(39, dtype=torch.int32, device="cuda")

    def run(i):
        y, dx, dw, db = torch.empty_like(i["dy"]), torch.empty_like(i["x"]), torch.empty_like(i["w"]), torch.empty(1024, device="cuda")
        rz.map_linear(i["x"], y, i["w"], act=2)
        rz.map_linear_grad(i["dy"], i["x"], i["w"], dx, dw, db, pre=y, act=1)
        n, dq, dg = torch.empty_like(i["q"]), torch.zeros_like(i["q"]), torch.empty(64, device="cuda")
        rz.map_qk_norm(i["q"], n, 4, 2, 64, row_pairs=16, col_pairs=16)
        rz.map_qk_norm_grad(n, i["q"], dq, 4, 2, 64, dgamma_q=dg, row_pairs=16, col_pairs=16)
        b, dt = torch.empty_like(i["s"]), torch.empty_like(i["t"])
        rz.map_position_bias(i["t"], lut, lut, b, (20, 20), (20, 20), scores=i["s"])
        rz.map_position_bias_grad(b, lut, lut, dt, (20, 20), (20, 20))
        return y, dx, dw, db, n, dq, dg, b, dt

    sets = [inputs(1), inputs(2)]
    alone = []
    for i in sets:
        alone.append(run(i))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(6):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(run(sets[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for outs in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(alone[k], outs))


def test_gradient_of_tiny_heads(rz):
    """Of heads of 1e-14 without eps: r^3 is past float32's range, the gradient is not."""
    x, dy = values((1, 2, 3, 64), "f32", 1, 1e-14), values((1, 2, 3, 64), "f32", 2)
    xv, dx = cuda(x), torch.empty((1, 2, 3, 64), device="cuda")
    rz.map_qk_norm_grad(cuda(dy), xv, dx, 1, 1, 32, eps=0.0, base=100.0, row_pairs=8, col_pairs=8)
    t = tok.angles(1, 2, 3, 32, None, 100.0, 8, 8, 1.0)
    want, _, _, e, _, _ = tok.qk_norm_grad(dy, x, 1, 1, 32, np.ones(32), np.ones(32), t, False, 0.0)
    check(dx, want, ref.stored(want, e, "f32"), "dx")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("act", [1, 2])
def test_slopes_of_infinite_sums(rz, dtype, act):
    """A pre past its type's range is infinite: the activation's slope there is 1 or 0."""
    dt = getattr(torch, tok.TORCH[dtype])
    pre = torch.tensor([np.inf, -np.inf, 3e4, -3e4], device="cuda").to(dt).view(1, 1, 1, 4)
    dy = torch.tensor([2.0, 2.0, -3.0, -3.0], device="cuda").to(dt).view(1, 1, 1, 4)
    x, w, db = torch.ones((1, 1, 1, 8), dtype=dt, device="cuda"), torch.ones((4, 8), dtype=dt, device="cuda"), torch.empty(4, device="cuda")
    rz.map_linear_grad(dy, x, w, dbias=db, pre=pre, act=act)
    assert db.cpu().tolist() == [2.0, 0.0, -3.0, 0.0]
    pre[..., 0] = float("nan")
    rz.map_linear_grad(dy, x, w, dbias=db, pre=pre, act=act)
    assert bool(torch.isnan(db[0])) and db[1:].cpu().tolist() == [0.0, -3.0, 0.0]


def test_weight_gradient_of_the_most_pixels(rz):
    """2^31 - 1 of them: the last 64 terms of the sum end at 2^31."""
    P, C = (1 << 31) - 1, 8
    torch.cuda.empty_cache()
    x, dy = (torch.zeros((1, 1, P, C), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # whole numbers at the beginning, in the middle and at the end: their sums are exact
    want = torch.zeros((C, C), dtype=torch.float64)
    rng = np.random.default_rng(3)
    for at in (0, 1 << 30, P - 130, P - 64):
        n = min(100, P - at)
        a, b = (torch.from_numpy(rng.integers(-8, 9, size=(n, C))).double() for _ in range(2))
        x[0, 0, at:at + n], dy[0, 0, at:at + n] = a.to("cuda", torch.bfloat16), b.to("cuda", torch.bfloat16)
    for at in (0, 1 << 30, P - 130):
        want += dy[0, 0, at:at + 130].double().cpu().T @ x[0, 0, at:at + 130].double().cpu()
    dw, db = torch.empty((C, C), device="cuda"), torch.empty(C, device="cuda")
    rz.map_linear_grad(dy, x, torch.zeros((C, C), dtype=torch.bfloat16, device="cuda"), None, dw, db)
    assert torch.equal(dw.double().cpu(), want)
    assert torch.equal(db.double().cpu(), sum(dy[0, 0, at:at + 130].double().cpu().sum(0) for at in (0, 1 << 30, P - 130)))
    del x, dy
    torch.cuda.empty_cache()
