"""The bilinear resize of channels-last maps and position tables, and its
gradient, against the 64-bit forms."""
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
    return ref.host(torch.from_numpy(np.random.default_rng(seed).normal(size=shape)).to(TYPES[dtype]))


def check_forward(rz, N, geo, C, dtype, table=False, src_dtype=None, base=True, slayout={}, layout={}, stream=None):
    H, W, OH, OW = geo
    src_dtype = src_dtype or dtype
    src, b = values((1 if table else N, H, W, C), src_dtype, 1), values((N, OH, OW, C), dtype, 2)
    sv, _ = ref.device_map(src, src_dtype, **slayout)
    bv = ref.device_map(b, dtype, **layout)[0] if base else None
    ov, flat = ref.device_map(np.zeros((N, OH, OW, C)), dtype, fill=-3.0, **layout)
    rz.resize_map(sv, ov, base=bv, stream=stream)
    torch.cuda.synchronize()
    up = ref.resize(src, OH, OW)
    want = up + (b if base else 0)
    # each weight and each of the three interpolations (a difference, a product and a sum) rounds: below 12 units
    # of the taps' size, and one for the added map
    err = ref.U * (12 * ref.resize(np.abs(src), OH, OW) + 12 * np.abs(up) + np.abs(want))
    err += ref.U * 8 * np.abs(src).max()
    assert np.all(np.abs(ref.host(ov) - want) <= ref.stored(want, err, dtype))
    assert ref.outside_untouched(flat, ov, -3.0)
    return ov


def check_gradient(rz, N, geo, C, dtype, table=False, src_dtype=None, slayout={}, layout={}, stream=None):
    H, W, OH, OW = geo
    src_dtype = src_dtype or dtype
    d = values((N, OH, OW, C), dtype, 3)
    dv, _ = ref.device_map(d, dtype, **layout)
    sv, flat = ref.device_map(np.zeros((1 if table else N, H, W, C)), src_dtype, fill=-3.0, **slayout)
    sv.fill_(7.0)
    rz.resize_map_grad(dv, sv, stream=stream)
    torch.cuda.synchronize()
    total = (lambda v: v.sum(0, keepdims=True)) if table else (lambda v: v)
    want, size = total(ref.resize_grad(d, H, W)), total(ref.resize_grad(np.abs(d), H, W))
    # roundings of the weights (4), of a product each way and of the sums, one for each image and reader
    terms = (N if table else 1) + 2 * (OH // H + 2) + 2 * (OW // W + 2)
    err = ref.U * (8 + terms) * size
    # a weight near 0 is off by half a unit of 1
    err += ref.U * 4 * total(np.abs(d).max() * np.ones_like(size)) * (N if table else 1)
    assert np.all(np.abs(ref.host(sv) - want) <= ref.stored(want, err, src_dtype))
    assert ref.outside_untouched(flat, sv, -3.0)


# doubled, halved, odd ratios, one-sample axes either way, unchanged, and a strong reduction that skips source pixels
GEOS = [(4, 6, 8, 12), (8, 12, 4, 6), (5, 7, 13, 10), (13, 10, 5, 7), (1, 1, 6, 5), (6, 5, 1, 1), (1, 9, 7, 3),
        (3, 3, 3, 3), (40, 33, 3, 4), (2, 3, 50, 41)]


@pytest.mark.parametrize("geo", GEOS)
@pytest.mark.parametrize("C", [1, 3, 8, 20, 64])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_maps(rz, geo, C, dtype):
    check_forward(rz, 2, geo, C, dtype, base=C % 2 == 0)
    check_gradient(rz, 2, geo, C, dtype)


@pytest.mark.parametrize("geo", [(6, 6, 9, 13), (9, 13, 6, 6), (5, 5, 5, 5)])
@pytest.mark.parametrize("dtype, src_dtype", [("bf16", "f32"), ("f16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("N, C", [(1, 16), (5, 24), (3, 7)])
def test_position_tables(rz, geo, dtype, src_dtype, N, C):
    check_forward(rz, N, geo, C, dtype, True, src_dtype)
    check_forward(rz, N, geo, C, dtype, True, src_dtype, base=False)
    check_gradient(rz, N, geo, C, dtype, True, src_dtype)


@pytest.mark.parametrize("layout", [dict(pad=8), dict(pad=16, gap=8), dict(gap=40), dict(offset=1), dict(pad=3)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_layouts(rz, layout, dtype):
    for table in (False, True):
        check_forward(rz, 2, (5, 6, 9, 11), 16, dtype, table, slayout=layout, layout=dict(layout, pad=24))
        check_gradient(rz, 2, (5, 6, 9, 11), 16, dtype, table, slayout=layout, layout=dict(layout, pad=24))


@pytest.mark.parametrize("geo, C, N", [((64, 48, 128, 96), 64, 3), ((100, 75, 61, 140), 40, 2), ((24, 24, 37, 50), 256, 6)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_larger_maps(rz, geo, C, N, dtype):
    for table in (False, True):
        check_forward(rz, N, geo, C, dtype, table)
        check_gradient(rz, N, geo, C, dtype, table)


def test_the_image_resize_of_three_channels(rz):
    # the plan's float resize of the same image: the same taps and weights
    img = torch.from_numpy(np.random.default_rng(6).random((37, 53, 3)) * 255).float().cuda()
    a, b = torch.empty((60, 41, 3), device="cuda"), torch.empty((60, 41, 3), device="cuda")
    rz.resize_map(img, a)
    with rz.resize_plan_create(37, 53, 60, 41, rz.RZ_LINEAR) as plan:
        rz.resize_f32(plan, img, b)
        torch.cuda.synchronize()
    assert float((a - b).abs().max()) <= 1e-4


def test_added_in_place(rz):
    src, base = (torch.from_numpy(values(s, "bf16", k)).bfloat16().cuda() for k, s in ((7, (1, 5, 5, 16)), (8, (3, 8, 9, 16))))
    want = torch.empty_like(base)
    rz.resize_map(src, want, base=base)
    rz.resize_map(src, base, base=base)
    assert torch.equal(base, want)


def test_gradient_against_differences(rz):
    # linear in the source: the forward of a direction is the difference
    v, d = values((2, 7, 5, 8), "f32", 9), values((2, 11, 12, 8), "f32", 10)
    vv, dv = ref.device_map(v, "f32")[0], ref.device_map(d, "f32")[0]
    out, g = torch.empty_like(dv), torch.empty_like(vv)
    rz.resize_map(vv, out)
    rz.resize_map_grad(dv, g)
    moved, product = (ref.host(out) * d).sum(), (ref.host(g) * v).sum()
    assert abs(moved - product) <= 64 * ref.U * np.abs(d).sum() * np.abs(v).max()


def test_not_a_number_stays_with_its_readers(rz):
    src = values((1, 6, 6, 8), "f32", 11)
    src[0, 2, 3, 4] = np.nan
    out = torch.empty((1, 12, 12, 8), device="cuda")
    rz.resize_map(ref.device_map(src, "f32")[0], out)
    reads = np.einsum("Y,X->YX", ref.axis_matrix(6, 12)[:, 2] > 0, ref.axis_matrix(6, 12)[:, 3] > 0)
    got = np.isnan(ref.host(out))
    assert np.all(got[0, :, :, 4][reads]) and not got[0, :, :, :4].any() and not got[0, :, :, 5:].any()


def test_empty_maps(rz):
    src = torch.ones((2, 4, 4, 8), device="cuda")
    for shape in [(2, 0, 3, 8), (2, 3, 0, 8)]:
        rz.resize_map(src, torch.empty(shape, device="cuda"))
        g = torch.ones_like(src)
        rz.resize_map_grad(torch.empty(shape, device="cuda"), g)
        assert bool((g == 0).all())
    g = torch.ones((1, 4, 4, 8), device="cuda")
    rz.resize_map_grad(torch.empty((0, 3, 3, 8), device="cuda"), g)
    assert bool((g == 0).all())
    rz.resize_map(torch.empty((0, 4, 4, 8), device="cuda"), torch.empty((0, 3, 3, 8), device="cuda"))
    rz.resize_map_grad(torch.empty((0, 3, 3, 8), device="cuda"), torch.empty((0, 4, 4, 8), device="cuda"))


def test_another_stream_and_a_graph(rz):
    s = torch.cuda.Stream()
    a = check_forward(rz, 3, (6, 6, 9, 13), 24, "bf16", True, "f32", stream=s)
    b = check_forward(rz, 3, (6, 6, 9, 13), 24, "bf16", True, "f32")
    assert torch.equal(a, b)
    check_gradient(rz, 3, (6, 6, 9, 13), 24, "bf16", True, "f32", stream=s.cuda_stream)
    d = torch.from_numpy(values((3, 9, 13, 24), "bf16", 12)).bfloat16().cuda()
    g = torch.empty((1, 6, 6, 24), device="cuda")
    ws = torch.empty(rz.resize_map_grad_workspace(d, g), dtype=torch.uint8, device="cuda")
    rz.resize_map_grad(d, g, workspace=ws)
    want = g.clone()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        rz.resize_map_grad(d, g, workspace=ws)
    g.zero_()
    ws.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g, want)


def test_offsets_past_32_bits(rz):
    # 2^31 elements and 2^32 bytes lie inside the output
    src = torch.empty((5, 512, 512, 512), dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.empty((5, 1024, 1024, 512), dtype=torch.bfloat16, device="cuda")
    rz.resize_map(src, out)
    one = torch.empty((1024, 1024, 512), dtype=torch.bfloat16, device="cuda")
    rz.resize_map(src[4], one)
    assert torch.equal(out[4], one)
    g, g1 = torch.empty_like(src), torch.empty_like(src[4])
    rz.resize_map_grad(out, g)
    rz.resize_map_grad(one, g1)
    assert torch.equal(g[4], g1)


def test_refusals(rz):
    src, dst = torch.zeros((2, 4, 4, 8), device="cuda"), torch.zeros((2, 6, 6, 8), device="cuda")
    flat = torch.zeros(1024, device="cuda")

    def arg(fn):
        with pytest.raises(rz.ResizeError) as e:
            fn()
        assert e.value.code == rz.RZ_ERR_ARG

    arg(lambda: rz.resize_map(src.half(), dst))
    arg(lambda: rz.resize_map(src, torch.empty((2, 70000, 1, 8), device="cuda")))
    arg(lambda: rz.resize_map(torch.empty((2, 0, 4, 8), device="cuda"), dst))
    arg(lambda: rz.resize_map(flat[:256].view(2, 4, 4, 8), flat[128:704].view(2, 6, 6, 8)))
    arg(lambda: rz.resize_map(src, flat[:576].view(2, 6, 6, 8), base=flat[8:584].view(2, 6, 6, 8)))
    arg(lambda: rz.resize_map_grad(flat[128:704].view(2, 6, 6, 8), flat[:256].view(2, 4, 4, 8)))
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    arg(lambda: rz.resize_map_grad(dst, src[:1], workspace=small))
    for call in (lambda: rz.resize_map(src[:, :, :, :4], dst), lambda: rz.resize_map(torch.zeros((3, 4, 4, 8), device="cuda"), dst),
                 lambda: rz.resize_map(src, dst, base=dst[:1]), lambda: rz.resize_map(src, dst, base=dst.half()),
                 lambda: rz.resize_map(src.permute(0, 3, 1, 2), dst), lambda: rz.resize_map(src.double(), dst)):
        with pytest.raises(ValueError):
            call()
