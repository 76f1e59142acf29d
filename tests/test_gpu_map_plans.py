"""The feature-map operators against the 64-bit forms where a call takes what
large ones do: clusters that go from unit to unit, joins of hundreds of chunks,
runs of rows with their readers on the way, means far above the deviation in
the pass kernels.  map_plans.py says which path each case takes."""
import numpy as np
import pytest

import map_plans as plans
import map_reference as ref
import test_gpu_map_norm as norm
import test_gpu_resize_map as resize

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rz():
    import __graft_entry__
    __graft_entry__.build()
    import bilinear_image_resize_gb300 as m
    torch.cuda.set_device(0)
    return m


def drop_factor(shape, p, seed, offset, first=0):
    """map_reference's drop_factor from block 0 on, all blocks at once in 64-bit integers."""
    assert first == 0
    t, total = ref.threshold(p), int(np.prod(shape))
    if t == 0:
        return np.ones(shape)
    word = np.uint64(0xFFFFFFFF)
    i = np.arange((total + 7) // 8, dtype=np.uint64)
    c = [i & word, i >> np.uint64(32), np.full_like(i, offset & 0xFFFFFFFF), np.full_like(i, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & word, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & word]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    lanes = np.stack([h for v in c for h in (v & np.uint64(0xFFFF), v >> np.uint64(16))], 1).reshape(-1)[:total]
    return np.where(lanes >= t, 65536 / (65536 - t) if t < 65536 else 0.0, 0.0).reshape(shape)


@pytest.fixture(autouse=True)
def fast(monkeypatch):
    slow = ref.drop_factor
    np.testing.assert_array_equal(drop_factor((5, 83), 0.3, (9 << 32) + 7, (3 << 32) + 2),
                                  slow((5, 83), 0.3, (9 << 32) + 7, (3 << 32) + 2))
    monkeypatch.setattr(ref, "drop_factor", drop_factor)


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("shape, G, dtype, grad", plans.ROUNDS_ALONE)
def test_units_of_single_ctas(rz, shape, G, dtype, grad, p):
    x = norm.features(shape, dtype, 21)
    (norm.check_gradient if grad else norm.check_forward)(rz, x, G, dtype, "silu", p)


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("shape, G, dtype, grad", plans.ROUNDS_CLUSTERS)
def test_units_of_clusters(rz, shape, G, dtype, grad, p):
    x = norm.features(shape, dtype, 22)
    (norm.check_gradient if grad else norm.check_forward)(rz, x, G, dtype, "silu" if p else "gelu", p)


@pytest.mark.parametrize("shape, G, dtype", plans.MANY_CHUNKS)
def test_many_chunks(rz, shape, G, dtype):
    x = norm.features(shape, dtype, 23)
    norm.check_forward(rz, x, G, dtype, "silu", 0.2)
    norm.check_gradient(rz, x, G, dtype, "silu", 0.2)


# padded rows; channels in no vector; an image that no cluster holds, in chunks of unlike lengths
@pytest.mark.parametrize("shape, G, layout", [((2, 30, 30, 32), 4, dict(pad=8)), ((2, 30, 30, 33), 3, {}),
                                              ((1, 200, 190, 32), 4, {})])
@pytest.mark.parametrize("offset", [300.0, -20000.0])
@pytest.mark.parametrize("first", [0.0, 1.0])
def test_mean_far_above_the_deviation_in_passes(rz, shape, G, layout, offset, first):
    assert layout or not plans.cluster_plans(shape, G, "f32", False)
    chunks, px, walk = plans.pass_plan(shape, 4 if shape[3] % 4 == 0 else 1, False)
    # the bound below counts at most 1024 roundings in a thread's own walk
    assert walk <= 1024 and (shape[1] < 200 or (chunks > 100 and shape[1] * shape[2] % px))
    x = np.random.default_rng(24).normal(size=shape) + offset
    x[:, 0, 0] *= first
    norm.check_forward(rz, x.astype(np.float32).astype(np.float64), G, "f32", "none", layout=layout)


@pytest.mark.parametrize("N, geo, C", plans.RESIZES)
@pytest.mark.parametrize("dtype", list(plans.SIZE))
def test_runs_of_rows(rz, N, geo, C, dtype):
    resize.check_forward(rz, N, geo, C, dtype, base=False)
    resize.check_gradient(rz, N, geo, C, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_runs_of_a_tables_rows(rz, dtype):
    resize.check_gradient(rz, *plans.TABLE, dtype, True, "f32")
