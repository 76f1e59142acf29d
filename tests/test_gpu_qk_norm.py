"""Norm of queries and keys with the position rotation, and its gradient, against
the 64-bit forms."""
import numpy as np
import pytest

import map_reference as ref
import token_reference as tok

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = ["f32", "bf16", "f16"]
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def values(shape, dtype, seed, scale=1.0):
    return tok.rounded(np.random.default_rng(seed).normal(size=shape) * scale, dtype)


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).float().cuda()


def check(got, want, bound, what):
    err = np.abs(ref.host(got) - want)
    assert np.all(err <= bound), (what, float((err / np.maximum(bound, 1e-300)).max()))


def both(rz, grid, heads, D, dtype, rows, cols, inter=False, positions=None, base=100.0, scale=1.0, more=0, layout={},
         affine=True, seed=1, in_place=False, parts="qk", **kw):
    """Forward and gradient; `more`: channels after the heads in x."""
    N, H, W = grid
    q, k = heads
    E = (q + k) * D
    x = values((N, H, W, E + more), dtype, seed)
    dy = values((N, H, W, E), dtype, seed + 1)
    gq, gk = (1 + values(D, "f32", seed + i, 0.3) if affine else np.ones(D) for i in (2, 3))
    gq, gk = tok.rounded(gq, "f32"), tok.rounded(gk, "f32")
    t = tok.angles(N, H, W, D, positions, base, rows, cols, scale)
    at = None if positions is None else torch.from_numpy(positions.astype(np.int32)).cuda()
    g = (cuda(gq), cuda(gk)) if affine else (None, None)
    turn = dict(positions=at, base=base, row_pairs=rows, col_pairs=cols, scale=scale, interleaved=inter)
    xv, _ = ref.device_map(x, dtype, **layout)
    yv, flat = ref.device_map(np.zeros((N, H, W, E)), dtype, fill=-3.0, **layout)
    stream = {k_: v for k_, v in kw.items() if k_ == "stream"}
    rz.map_qk_norm(xv, yv, q, k, D, *g, **turn, **stream)
    torch.cuda.synchronize()
    want, err = tok.qk_norm(x, q, k, D, gq, gk, t, inter, EPS)
    check(yv, want, ref.stored(want, err, dtype), "y")
    assert ref.outside_untouched(flat, yv, -3.0)
    if in_place:
        zv, zflat = ref.device_map(x, dtype, fill=-3.0, **layout)
        rz.map_qk_norm(zv, zv, q, k, D, *g, **turn)
        assert torch.equal(zv[..., :E], yv)
        assert np.array_equal(ref.host(zv)[..., E:], x[..., E:]) and ref.outside_untouched(zflat, zv, -3.0)
    dv, _ = ref.device_map(dy, dtype, **layout)
    ov, oflat = ref.device_map(np.full(x.shape, 4.0), dtype, fill=-3.0, **layout)
    dq, dk = (torch.full((D,), 9.0, device="cuda") for _ in range(2))
    rz.map_qk_norm_grad(dv, xv, ov, q, k, D, *g, dq if "q" in parts else None, dk if "k" in parts else None, **turn, **kw)
    torch.cuda.synchronize()
    dx, wq, wk, ex, eq, ek = tok.qk_norm_grad(dy, x, q, k, D, gq, gk, t, inter, EPS)
    check(ov[..., :E], dx, ref.stored(dx, ex, dtype), "dx")
    assert bool((ov[..., E:] == 4.0).all()) and ref.outside_untouched(oflat, ov, -3.0)
    if "q" in parts:
        check(dq, wq, eq + 2.0 ** -24 * np.abs(wq), "dgamma_q")
    if "k" in parts:
        check(dk, wk, ek + 2.0 ** -24 * np.abs(wk), "dgamma_k")
    return yv, ov, dq, dk


# every way a head is shared out: one pair, odd halves, vectors of four, groups that fill no power of two, the largest
@pytest.mark.parametrize("D", [2, 6, 8, 24, 32, 40, 64, 72, 80, 96, 128, 200, 254, 256])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_head_sizes(rz, D, inter, dtype):
    rows = D // 4
    both(rz, (2, 3, 5), (3, 2), D, dtype, rows, D // 2 - rows, inter, more=D)


# no rotation, some pairs that stay, one kind of heads only, many heads, one token
@pytest.mark.parametrize("heads", [(1, 0), (0, 1), (5, 5), (16, 1), (33, 11)])
@pytest.mark.parametrize("rows, cols", [(0, 0), (0, 16), (16, 0), (5, 7)])
@pytest.mark.parametrize("grid", [(1, 1, 1), (2, 1, 37), (3, 9, 1)])
def test_heads_and_pairs(rz, heads, rows, cols, grid):
    both(rz, grid, heads, 32, "bf16", rows, cols, more=32 if heads[0] % 2 else 0)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("base, scale", [(10000.0, 1.0), (500000.0, 0.125), (100.0, 9.0), (10.0, -1.0)])
def test_far_positions(rz, inter, dtype, base, scale):
    rng = np.random.default_rng(5)
    p = rng.integers(-(1 << 31), 1 << 31, size=(2, 3, 5, 2))
    p[0] = rng.integers(0, 1 << 20, size=(3, 5, 2))
    p[1, 0, 0] = (-(1 << 31), (1 << 31) - 1)
    p[1, 0, 1] = 0
    # base^(-j / n) and the step's turn in float64: 4 units of 2^-53 of an angle of up to 2^31 scale radians, 1e-6 scale, which the
    # bound's 6 units of a cosine do not cover: positions of this test stay where it is below a unit
    p = np.sign(p) * (np.abs(p) >> (10 if abs(scale) <= 1 else 14))
    both(rz, (2, 3, 5), (4, 2), 64, dtype, 13, 19, inter, positions=p, base=base, scale=scale)


def test_whole_turns_of_any_int(rz):
    """A step of an eighth of a turn, which 2^64 divides: every int lands on one of eight angles."""
    D = 8
    p = np.array([-(1 << 31), (1 << 31) - 1, -1, 0, 1, 7, 8, (1 << 24) + 3]).reshape(1, 1, 8, 1) * np.ones(2, np.int64)
    x = values((1, 1, 8, D), "f32", 3)
    y = torch.empty((1, 1, 8, D), device="cuda")
    at = torch.from_numpy(p.astype(np.int32)).cuda()
    rz.map_qk_norm(cuda(x), y, 1, 0, D, positions=at, base=1.0, row_pairs=2, col_pairs=2, scale=2 * np.pi / 8)
    t = np.zeros((1, 1, 8, 1, 4)) + (p[..., :1, None] % 8) * np.pi / 4
    want, err = tok.qk_norm(x, 1, 0, D, np.ones(D), np.ones(D), t, False, EPS)
    # the step's own rounding, 2^-53 of it, times 2^31 positions
    check(y, want, err + 2.0 ** -22 * tok.pair_sum(want, False), "y")


LAYOUTS = [dict(pad=16), dict(gap=64), dict(pad=8, gap=24), dict(offset=1), dict(pad=4, offset=4), dict(pad=1)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("more", [0, 32, 3])
def test_layouts(rz, layout, dtype, more):
    both(rz, (2, 3, 7), (2, 1), 32, dtype, 8, 8, layout=layout, more=more, in_place=True)


@pytest.mark.parametrize("parts", ["q", "k", ""])
def test_parts_and_no_gammas(rz, parts):
    both(rz, (2, 5, 7), (3, 2), 64, "f16", 16, 16, affine=False, parts=parts)
    both(rz, (2, 5, 7), (3, 2), 64, "f16", 16, 16, parts=parts)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("grid, heads, D", [((3, 48, 50), (4, 4), 64), ((1, 70, 90), (16, 2), 32), ((2, 30, 31), (2, 2), 72)])
def test_larger(rz, dtype, grid, heads, D):
    both(rz, grid, heads, D, dtype, D // 4, D // 2 - D // 4, more=D * heads[1])


def test_gradient_in_place(rz):
    x, dy = values((2, 3, 5, 96), "bf16", 1), values((2, 3, 5, 96), "bf16", 2)
    xv, dv = (torch.from_numpy(a).bfloat16().cuda() for a in (x, dy))
    out = torch.empty_like(xv)
    rz.map_qk_norm_grad(dv, xv, out, 1, 1, 32, base=10.0, row_pairs=8)
    rz.map_qk_norm_grad(dv, xv, dv, 1, 1, 32, base=10.0, row_pairs=8)
    assert torch.equal(dv[..., :64], out[..., :64]) and np.array_equal(ref.host(dv)[..., 64:], dy[..., 64:])


def test_heads_of_zeros(rz):
    x = torch.zeros((1, 2, 2, 64), device="cuda")
    x[0, 0, 0, 32:] = 1.0
    y = torch.full_like(x, 5.0)
    rz.map_qk_norm(x, y, 1, 1, 32)
    assert float(y[..., :32].abs().max()) == 0 and float(y[0, 1].abs().max()) == 0
    dx, dg = torch.full_like(x, 5.0), torch.full((32,), 5.0, device="cuda")
    rz.map_qk_norm_grad(torch.ones_like(x), x, dx, 1, 1, 32, dgamma_q=dg)
    assert bool(torch.isfinite(dx).all()) and float(dg.abs().max()) == 0


def test_empty_maps(rz):
    for shape in ((0, 3, 3, 64), (2, 0, 3, 64)):
        x = torch.empty(shape, device="cuda")
        dg = torch.full((32,), 5.0, device="cuda")
        rz.map_qk_norm(x, torch.empty_like(x), 1, 1, 32)
        rz.map_qk_norm_grad(x, x, torch.empty_like(x), 1, 1, 32, dgamma_k=dg)
        assert float(dg.abs().max()) == 0


def test_same_bits_other_stream_given_workspace(rz):
    first = [t.clone() for t in both(rz, (3, 20, 21), (4, 2), 64, "f16", 16, 16)]
    x, dy = torch.empty((3, 20, 21, 384), dtype=torch.float16, device="cuda"), torch.empty((3, 20, 21, 384), dtype=torch.float16, device="cuda")
    n = rz.map_qk_norm_grad_workspace(dy, x, 4, 2, 64)
    work = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = both(rz, (3, 20, 21), (4, 2), 64, "f16", 16, 16, workspace=work[:n], stream=s)
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and bool((work[n:] == 0xA5).all())


def test_captured_and_replayed(rz):
    grid, D = (2, 6, 9), 64
    x, dy = (torch.zeros((*grid, 3 * D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    dq, dk = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    work = torch.empty(rz.map_qk_norm_grad_workspace(dy, x, 2, 1, D), dtype=torch.uint8, device="cuda")

    def step():
        rz.map_qk_norm(x, y, 2, 1, D, base=50.0, row_pairs=16)
        rz.map_qk_norm_grad(dy, x, dx, 2, 1, D, None, None, dq, dk, base=50.0, row_pairs=16, workspace=work)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    t = tok.angles(*grid, D, None, 50.0, 16, 16, 1.0)
    for seed in (1, 2):
        vx, vd = values(tuple(x.shape), "bf16", seed), values(tuple(x.shape), "bf16", seed + 9)
        x.copy_(torch.from_numpy(vx))
        dy.copy_(torch.from_numpy(vd))
        g.replay()
        torch.cuda.synchronize()
        one = np.ones(D)
        want, err = tok.qk_norm(vx, 2, 1, D, one, one, t, False, EPS)
        check(y, want, ref.stored(want, err, "bf16"), "y")
        gx, wq, wk, ex, eq, ek = tok.qk_norm_grad(vd, vx, 2, 1, D, one, one, t, False, EPS)
        check(dx, gx, ref.stored(gx, ex, "bf16"), "dx")
        check(dq, wq, eq + 1e-7 * np.abs(wq), "dgamma_q")
        check(dk, wk, ek + 1e-7 * np.abs(wk), "dgamma_k")


def test_gradient_against_differences(rz):
    grid, heads, D, h = (2, 3, 4), (2, 1), 24, 2.0 ** -7
    x, dy = values((*grid, 72), "f32", 1), values((*grid, 72), "f32", 2)
    gq = 1 + values(D, "f32", 3, 0.2)
    turn = dict(base=20.0, row_pairs=5, col_pairs=6, interleaved=True)
    dx, dg = torch.empty((*grid, 72), device="cuda"), torch.empty(D, device="cuda")
    rz.map_qk_norm_grad(cuda(dy), cuda(x), dx, *heads, D, cuda(gq), None, dg, **turn)
    rng = np.random.default_rng(7)
    for k, g in ((0, dx), (1, dg)):
        d = rng.normal(size=(x, gq)[k].shape)
        d /= np.linalg.norm(d)
        sums = []
        for s in (1, -1):
            a = [x, gq]
            a[k] = tok.rounded(a[k] + s * h * d, "f32")
            y = torch.empty((*grid, 72), device="cuda")
            rz.map_qk_norm(cuda(a[0]), y, *heads, D, cuda(a[1]), **turn)
            sums.append(float((ref.host(y) * dy).sum()))
        slope = (sums[0] - sums[1]) / (2 * h)
        # 25 U of each |y| before the division by 2 h, six deviations of the sum; a smooth sum's third derivative, 1e-3
        noise = 6 * 25 * 2.0 ** -24 * np.linalg.norm(ref.host(y) * dy) / h + 1e-3 * np.linalg.norm(ref.host(g))
        assert abs(slope - float((ref.host(g) * d).sum())) <= noise


# a few hundred tokens, whose heads are cut into runs that no whole number of warps takes: a warp's second item is another
# token's run (the cut into whole runs once left empty ones, after which the gradient read vectors of another step)
@pytest.mark.parametrize("grid, heads, D, dtype", [((1, 16, 16), (12, 12), 128, "f32"), ((1, 30, 30), (2, 2), 256, "f32"),
                                                   ((1, 14, 14), (16, 16), 128, "f32"), ((2, 12, 12), (32, 8), 64, "f32"),
                                                   ((1, 17, 17), (32, 8), 128, "bf16"), ((1, 14, 14), (16, 16), 256, "bf16"),
                                                   ((1, 16, 16), (16, 16), 256, "f16"), ((1, 16, 18), (20, 20), 128, "f16"),
                                                   ((3, 8, 17), (4, 3), 24, "f16"), ((2, 19, 16), (5, 2), 100, "f32")])
@pytest.mark.parametrize("inter", [False, True])
def test_some_hundred_tokens(rz, grid, heads, D, dtype, inter):
    first = both(rz, grid, heads, D, dtype, D // 4, D // 2 - D // 4, inter)
    again = both(rz, grid, heads, D, dtype, D // 4, D // 2 - D // 4, inter)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("base, scale", [(10000.0, 1.0), (500000.0, 9.0), (100.0, -1000.0), (10.0, 0.125)])
def test_any_int_position(rz, dtype, base, scale):
    """The whole range of int, and steps of many turns: the angle is good to 2^-24 of half a turn all the same."""
    N, H, W, q, k, D, rows = 2, 3, 8, 2, 1, 32, 7
    rng = np.random.default_rng(11)
    p = rng.integers(-(1 << 31), 1 << 31, size=(N, H, W, 2))
    p[0, 0, 0], p[0, 0, 1], p[0, 0, 2] = (-(1 << 31), (1 << 31) - 1), ((1 << 31) - 1, -(1 << 31)), (0, -1)
    x, dy = values((N, H, W, 96), dtype, 1), values((N, H, W, 96), dtype, 2)
    xv, dv = (torch.from_numpy(a).to(getattr(torch, tok.TORCH[dtype])).cuda() for a in (x, dy))
    y, dx, dq = torch.empty_like(xv), torch.empty_like(xv), torch.empty(D, device="cuda")
    turn = dict(positions=torch.from_numpy(p.astype(np.int32)).cuda(), base=base, row_pairs=rows, scale=scale)
    rz.map_qk_norm(xv, y, q, k, D, **turn)
    rz.map_qk_norm_grad(dv, xv, dx, q, k, D, dgamma_q=dq, **turn)
    t = tok.exact_angles(N, H, W, D, p, base, rows, D // 2 - rows, scale)
    one = np.ones(D)
    want, err = tok.qk_norm(x, q, k, D, one, one, t, False, EPS)
    gx, gq, _, ex, eq, _ = tok.qk_norm_grad(dy, x, q, k, D, one, one, t, False, EPS)
    if dtype != "f32":      # 16-bit maps' cosines and sines: 7e-7, six units of 2^-24 more than the bounds have
        more = 6 * 2.0 ** -24
        r = 1 / np.sqrt((x.reshape(N, H, W, 3, D) ** 2).mean(-1, keepdims=True) + EPS)
        spread = tok.pair_sum(dy.reshape(N, H, W, 3, D), False)
        h = np.abs(x.reshape(N, H, W, 3, D) * r)
        err = err + more * tok.pair_sum((x.reshape(N, H, W, 3, D) * r), False).reshape(err.shape)
        ex = ex + more * (r * spread + r * h * (spread * h).mean(-1, keepdims=True)).reshape(ex.shape)
        eq = eq + more * (spread * h)[..., :q, :].sum((0, 1, 2, 3))
    check(y, want, ref.stored(want, err, dtype), "y")
    check(dx, gx, ref.stored(gx, ex, dtype), "dx")
    check(dq, gq, eq + 2.0 ** -24 * np.abs(gq), "dgamma_q")
