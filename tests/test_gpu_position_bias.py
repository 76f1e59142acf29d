"""Relative position bias by buckets, and the gradient of its table, against the
64-bit forms."""
import numpy as np
import pytest

import map_reference as ref
import token_reference as tok

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

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


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def matrices(a, dtype, pad=0, gap=0, offset=0, fill=0.0):
    """(N, heads, q, k): `pad` elements after each row, `gap` after each head's matrix."""
    N, h, q, k = a.shape
    view, flat = ref.device_map(a.reshape(N * h, q, 1, k), dtype, pad, gap, offset, fill)
    s = view.stride()
    return torch.as_strided(flat, a.shape, (h * s[0], s[0], s[1], 1), offset), flat


def both(rz, N, heads, query, key, dtype, rule=(4, 6, 20), shift=(0, 0), scores=True, layout={}, seed=1, in_place=False,
         luts=None, **kw):
    R = 2 * rule[1] - 1
    rows, cols = luts or (tok.buckets(query[0], key[0], *rule, shift[0]), tok.buckets(query[1], key[1], *rule, shift[1]))
    table = values((R, R, heads), "f32", seed)
    shape = (N, heads, query[0] * query[1], key[0] * key[1])
    bias = tok.position_bias(table, rows, cols, query, key)
    t, r, c = cuda(table).float(), cuda(rows.astype(np.int32)), cuda(cols.astype(np.int32))
    s = values(shape, dtype, seed + 1, 3.0)
    if scores and s.size > 8:
        s[..., shape[3] // 2] = -np.inf                       # a masked key
        s[:, 0, 0] = -np.inf                                  # a row that sees nothing
        low = float(torch.finfo(getattr(torch, tok.TORCH[dtype])).min)
        s[:, -1, -1, : max(1, shape[3] // 3)] = low           # masks of the type's lowest value
    want = (s if scores else 0) + np.broadcast_to(bias, shape)
    out, flat = matrices(s if in_place else np.zeros(shape), dtype, fill=-3.0, **layout)
    sv = out if in_place else matrices(s, dtype, **layout)[0] if scores else None
    stream = {k: v for k, v in kw.items() if k == "stream"}
    rz.map_position_bias(t, r, c, out, query, key, scores=sv, **stream)
    torch.cuda.synchronize()
    got = ref.host(out)
    lowest = float(torch.finfo(out.dtype).min)
    masked = np.isinf(want) | (want <= lowest)
    # a lowest value and a bias round to it, or past it to -infinity where the bias is more than half a step
    half = abs(lowest) * float(torch.finfo(out.dtype).eps) / 4
    finite = ~masked
    assert np.array_equal(np.isneginf(got[np.isinf(want)]), np.ones(int(np.isinf(want).sum()), bool))
    edge = masked & ~np.isinf(want)
    assert np.all(np.where(want[edge] < lowest - half, np.isneginf(got[edge]) | (got[edge] == lowest), got[edge] == lowest))
    err = np.abs(got[finite] - want[finite])
    assert np.all(err <= ref.stored(want[finite], 2.0 ** -24 * np.abs(want[finite]), dtype))
    assert ref.outside_untouched(flat, out, -3.0)

    d = values(shape, dtype, seed + 2)
    dv, _ = matrices(d, dtype, **layout)
    dt = torch.full((R, R, heads), 9.0, device="cuda")
    rz.map_position_bias_grad(dv, r, c, dt, query, key, **kw)
    torch.cuda.synchronize()
    w, mag, count = tok.position_bias_grad(d, rows, cols, query, key, R, R)
    steps = np.vectorize(ref.walk)(np.maximum(count, 1))[..., None]
    err = np.abs(ref.host(dt) - w)
    assert np.all(err <= 2.0 ** -24 * (steps * mag + np.abs(w))), float(err.max())
    assert np.all(ref.host(dt)[count == 0] == 0)
    return out, dt


# one query, one key; a row, a column; windows; grids of different sizes; rows wider than a tile, taller than one
GRIDS = [((1, 1), (1, 1)), ((1, 1), (3, 5)), ((1, 7), (1, 9)), ((6, 1), (11, 1)), ((7, 7), (7, 7)), ((8, 8), (8, 8)),
         ((3, 5), (6, 10)), ((6, 10), (3, 5)), ((5, 3), (2, 16)), ((70, 2), (67, 3)), ((2, 3), (3, 300)), ((1, 90), (1, 150)),
         ((66, 1), (1, 5)), ((20, 24), (20, 24))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("query, key", GRIDS)
@pytest.mark.parametrize("N, heads", [(1, 3), (2, 1)])
def test_grids(rz, query, key, dtype, N, heads):
    both(rz, N, heads, query, key, dtype)
    both(rz, N, heads, query, key, dtype, scores=False)


# a large batch of small matrices
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [7, 8, 9, 100])
@pytest.mark.parametrize("query, key", [((7, 7), (7, 7)), ((4, 4), (4, 6)), ((1, 1), (2, 3)), ((1, 1), (40, 50))])
def test_batches(rz, N, query, key, dtype):
    both(rz, N, 4, query, key, dtype)


@pytest.mark.parametrize("rule", [(1, 1, 2), (1, 2, 3), (3, 3, 5), (8, 16, 128), (2, 9, 40), (16, 32, 33)])
@pytest.mark.parametrize("shift", [(0, 0), (5, -3)])
def test_rules(rz, rule, shift):
    both(rz, 1, 2, (9, 12), (13, 11), "f32", rule, shift)


LAYOUTS = [dict(pad=16), dict(gap=64), dict(pad=7), dict(offset=1), dict(pad=3, gap=5, offset=2), dict(pad=8, offset=8)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N, query, key", [(2, (5, 8), (5, 8)), (9, (3, 3), (3, 3)), (2, (1, 20), (1, 33)), (60, (3, 3), (3, 3))])
def test_layouts(rz, layout, dtype, N, query, key):
    both(rz, N, 2, query, key, dtype, layout=layout)
    both(rz, N, 2, query, key, dtype, layout=layout, in_place=True)


@pytest.mark.parametrize("N", [1, 9, 60])
def test_scores_that_begin_elsewhere_in_their_vectors(rz, N):
    query = key = (5, 8)
    rule = (4, 6, 20)
    rows = tok.buckets(5, 5, *rule)
    cols = tok.buckets(8, 8, *rule)
    table, s = values((11, 11, 2), "f32", 1), values((N, 2, 40, 40), "bf16", 2)
    sv, out = matrices(s, "bf16", offset=3)[0], matrices(np.zeros(s.shape), "bf16")[0]
    rz.map_position_bias(cuda(table).float(), cuda(rows), cuda(cols), out, query, key, scores=sv)
    want = s + tok.position_bias(table, rows, cols, query, key)
    assert np.all(np.abs(ref.host(out) - want) <= ref.stored(want, 2.0 ** -24 * np.abs(want), "bf16"))


@pytest.mark.parametrize("N", [1, 9, 40])
def test_buckets_outside_the_table_have_no_bias(rz, N):
    rng = np.random.default_rng(3)
    rows, cols = rng.integers(-3, 14, 6 + 5 - 1), rng.integers(-3, 14, 4 + 7 - 1)
    rows[0], cols[2] = (1 << 31) - 1, -(1 << 31)
    both(rz, N, 3, (6, 4), (5, 7), "f32", (6, 6, 7), luts=(rows, cols))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N, heads, query, key", [(1, 2, (40, 44), (40, 44)), (2, 3, (1, 1500), (1, 1500)),
                                                  (300, 3, (7, 7), (7, 7)), (1, 1, (1, 1), (200, 300)),
                                                  (1, 1, (2100, 1), (2100, 1))])
def test_larger(rz, dtype, N, heads, query, key):
    both(rz, N, heads, query, key, dtype, (8, 16, 128))


def test_same_bits_other_stream_given_workspace(rz):
    first = [t.clone() for t in both(rz, 3, 2, (20, 24), (20, 24), "bf16")]
    d, t = torch.empty((3, 2, 480, 480), dtype=torch.bfloat16, device="cuda"), torch.empty((11, 11, 2), device="cuda")
    n = rz.map_position_bias_grad_workspace(d, t, (20, 24), (20, 24))
    work = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = both(rz, 3, 2, (20, 24), (20, 24), "bf16", workspace=work[:n], stream=s)
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and bool((work[n:] == 0xA5).all())


def test_captured_and_replayed(rz):
    query = key = (6, 8)
    rule, shape = (3, 5, 9), (2, 3, 48, 48)
    rows, cols = tok.buckets(6, 6, *rule), tok.buckets(8, 8, *rule)
    r, c = cuda(rows), cuda(cols)
    table, s = torch.zeros((9, 9, 3), device="cuda"), torch.zeros(shape, dtype=torch.float16, device="cuda")
    out, dt = torch.zeros_like(s), torch.zeros_like(table)
    work = torch.empty(rz.map_position_bias_grad_workspace(s, dt, query, key), dtype=torch.uint8, device="cuda")

    def step():
        rz.map_position_bias(table, r, c, out, query, key, scores=s)
        rz.map_position_bias_grad(s, r, c, dt, query, key, workspace=work)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        vt, vs = values((9, 9, 3), "f32", seed), values(shape, "f16", seed + 4)
        table.copy_(torch.from_numpy(vt))
        s.copy_(torch.from_numpy(vs))
        g.replay()
        torch.cuda.synchronize()
        want = vs + tok.position_bias(vt, rows, cols, query, key)
        assert np.all(np.abs(ref.host(out) - want) <= ref.stored(want, 2.0 ** -24 * np.abs(want), "f16"))
        w, mag, count = tok.position_bias_grad(vs, rows, cols, query, key, 9, 9)
        assert np.all(np.abs(ref.host(dt) - w) <= 2.0 ** -24 * (np.vectorize(ref.walk)(np.maximum(count, 1))[..., None] * mag + np.abs(w)))


def test_empty(rz):
    t, i = torch.full((3, 3, 2), 5.0, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    d = torch.empty((0, 2, 4, 9), device="cuda")
    rz.map_position_bias(t, i, i, d, (2, 2), (3, 3))
    rz.map_position_bias_grad(d, i, i, t, (2, 2), (3, 3))
    assert float(t.abs().max()) == 0


def test_gradient_against_differences(rz):
    """The bias is linear in the table: one step shows the slope up to float32's rounding."""
    query = key = (4, 5)
    rule = (2, 4, 6)
    r, c = cuda(tok.buckets(4, 4, *rule)), cuda(tok.buckets(5, 5, *rule))
    d, step = values((2, 3, 20, 20), "f32", 1), values((7, 7, 3), "f32", 2)
    out, dt = torch.empty((2, 3, 20, 20), device="cuda"), torch.empty((7, 7, 3), device="cuda")
    rz.map_position_bias(cuda(step).float(), r, c, out, query, key)
    rz.map_position_bias_grad(cuda(d).float(), r, c, dt, query, key)
    want = float((ref.host(out) * d).sum())
    assert abs(float((ref.host(dt) * step).sum()) - want) <= 2.0 ** -24 * 64 * float(np.abs(ref.host(out) * d).sum())
