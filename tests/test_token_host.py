"""Host-side checks of the operators around attention: arguments refused before
any CUDA call, struct layouts, workspace sizes, buckets.  No GPU needed."""
import ctypes
import os
import random

import numpy as np
import pytest

import token_reference as tok
from conftest import ROOT

ARG, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from bilinear_image_resize_gb300 import _build, _native
    _build.build()
    return _native.load()


@pytest.fixture(scope="module")
def nat():
    from bilinear_image_resize_gb300 import _native
    return _native


@pytest.mark.parametrize("cname, pyname", [("rz_linear", "RzLinear"), ("rz_qk", "RzQk"), ("rz_bias", "RzBias")])
def test_struct_layouts_match_header(tmp_path, nat, cname, pyname):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    cls = getattr(nat, pyname)
    fields = [f[0] for f in cls._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "gbresize.h"\nint main(void){'
                    f'printf("%zu", sizeof({cname}));' +
                    "".join(f'printf(" %zu", offsetof({cname}, {n}));' for n in fields) + "return 0;}\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(tmp_path / "a")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, n).offset for n in fields]


def test_linear_refuses(lib, nat):
    good = dict(N=2, H=4, W=4, C=16, K=24, dtype=2, act=0)
    x, y, other = nat.RzMap(1 << 20, 128, 512), nat.RzMap(1 << 21, 192, 768), nat.RzMap(1 << 22, 192, 768)
    w, n, ws = 1 << 23, ctypes.c_size_t(7), 1 << 30

    def query(x=x, w=w, pitch=32, r=None, pre=None, y=y, out=n, **change):
        return lib.map_linear_workspace(nat.RzLinear(**{**good, **change}), x, w, pitch, r, pre, y,
                                        None if out is None else ctypes.byref(out))

    def call(x=x, w=w, pitch=32, b=None, r=None, pre=None, y=y, work=ws, size=1 << 30, status=None, **change):
        return lib.map_linear(nat.RzLinear(**{**good, **change}), x, w, pitch, b, r, pre, y, work, size, status, None)

    assert query() == 0 and n.value == 0                      # aligned 16-bit maps are read and written where they lie
    assert query(N=1, H=2, W=4, x=nat.RzMap((1 << 20) + 2, 128, 512)) == 0 and n.value == 0    # eight pixels
    assert query(N=3, dtype=1, x=nat.RzMap(1 << 20, 256, 1024), y=nat.RzMap(1 << 21, 384, 1536), pitch=64) == 0 and n.value >= 6 * 16 * (48 + 24)
    assert lib.map_linear_workspace(None, x, w, 32, None, None, y, ctypes.byref(n)) == ARG and query(out=None) == ARG
    for change in (dict(N=-1), dict(H=-1), dict(C=0), dict(K=0), dict(C=65537), dict(K=65537), dict(dtype=0), dict(dtype=4),
                   dict(act=-1), dict(act=3), dict(x=None), dict(y=None), dict(w=None), dict(w=w + 1), dict(pitch=30), dict(pitch=33),
                   dict(x=nat.RzMap((1 << 20) + 1, 128, 512)), dict(x=nat.RzMap(1 << 20, 126, 512)),
                   dict(y=nat.RzMap(1 << 21, 192, 760)), dict(r=nat.RzMap(1 << 22, 190, 768)), dict(pre=nat.RzMap((1 << 22) + 1, 192, 768)),
                   dict(H=1 << 16, W=1 << 15)):
        assert query(**change) == ARG and call(**change) == ARG, change
    big = dict(N=1 << 16, H=1 << 8, W=1 << 8, C=1, K=1, pitch=2)
    assert query(x=nat.RzMap(1 << 40, 512, 1 << 17), y=nat.RzMap(1 << 50, 512, 1 << 17), **big) == UNSUPPORTED
    # overlaps: y with x, weight, bias, another residual; pre with anything
    for change in (dict(y=nat.RzMap((1 << 20) + 512, 192, 768)), dict(w=(1 << 21) + 64), dict(b=(1 << 21) + 64),
                   dict(r=nat.RzMap((1 << 21) + 192, 192, 768)), dict(pre=y), dict(pre=nat.RzMap((1 << 20) + 16, 192, 768)),
                   dict(pre=other, r=other), dict(pre=other, w=(1 << 22) + 16), dict(pre=other, b=(1 << 22) + 16), dict(b=2), dict(status=2)):
        assert call(**change) == ARG, change
    # float32 needs a workspace: none, misaligned, too small
    f = dict(N=3, dtype=1, x=nat.RzMap(1 << 20, 256, 1024), y=nat.RzMap(1 << 21, 384, 1536), pitch=64)
    assert call(work=None, **f) == ARG and call(work=ws + 8, **f) == ARG and call(size=64, **f) == ARG
    empty = nat.RzLinear(**{**good, "N": 0})
    assert lib.map_linear(empty, None, None, 0, None, None, None, None, None, 0, None, None) == 0
    assert lib.map_linear_workspace(empty, None, None, 0, None, None, None, ctypes.byref(n)) == 0 and n.value == 0


def test_linear_grad_refuses(lib, nat):
    good = dict(N=2, H=4, W=4, C=16, K=24, dtype=2, act=1)
    x, dy, pre, dx = nat.RzMap(1 << 20, 128, 512), nat.RzMap(1 << 21, 192, 768), nat.RzMap(1 << 22, 192, 768), nat.RzMap(1 << 24, 128, 512)
    w, dw, db, n, ws = 1 << 23, 1 << 25, 1 << 26, ctypes.c_size_t(7), 1 << 30

    def query(dy=dy, x=x, w=w, pitch=32, pre=pre, dx=dx, dw=dw, dp=32, dt=2, out=n, **change):
        return lib.map_linear_grad_workspace(nat.RzLinear(**{**good, **change}), dy, x, w, pitch, pre, dx, dw, dp, dt,
                                             None if out is None else ctypes.byref(out))

    def call(dy=dy, x=x, w=w, pitch=32, pre=pre, dx=dx, dw=dw, dp=32, dt=2, db=db, work=ws, size=1 << 30, **change):
        return lib.map_linear_grad(nat.RzLinear(**{**good, **change}), dy, x, w, pitch, pre, dx, dw, dp, dt, db, work, size, None, None)

    assert query() == 0 and n.value >= 32 * 48
    whole = n.value
    assert query(dx=None, dw=None) == 0 and n.value < whole
    assert query(out=None) == ARG
    for change in (dict(dy=None), dict(x=None), dict(w=None), dict(pre=None), dict(dt=3), dict(dt=0), dict(dp=30), dict(dp=33), dict(dw=dw + 1),
                   dict(act=4), dict(K=0), dict(dx=nat.RzMap(1 << 24, 126, 512)), dict(pre=nat.RzMap(1 << 22, 191, 768))):
        assert query(**change) == ARG and call(**change) == ARG, change
    assert query(act=0, pre=None) == 0
    assert query(dt=1, dp=64) == 0 and query(dt=1, dp=32) == ARG
    for change in (dict(dx=dy), dict(dx=x), dict(dx=nat.RzMap((1 << 21) + 256, 128, 512)), dict(dx=nat.RzMap((1 << 22) + 256, 128, 512)),
                   dict(dw=1 << 23), dict(dw=(1 << 20) + 32), dict(db=(1 << 24) + 16), dict(db=(1 << 25) + 16), dict(db=2), dict(work=None),
                   dict(work=ws + 4), dict(size=100)):
        assert call(**change) == ARG, change


def test_qk_norm_refuses(lib, nat):
    good = dict(N=2, H=4, W=4, C=96, out_C=64, q_heads=1, k_heads=1, D=32, dtype=2, row_pairs=8, col_pairs=8, interleaved=0, eps=1e-6,
                base=100.0, scale=1.0)
    x, y = nat.RzMap(1 << 20, 768, 3840), nat.RzMap(1 << 21, 512, 2048)
    n, ws = ctypes.c_size_t(7), 1 << 30

    def call(x=x, y=y, gq=None, gk=None, at=None, **change):
        return lib.map_qk_norm(nat.RzQk(**{**good, **change}), x, y, gq, gk, at, None)

    def grad(dy=y, x=x, dx=nat.RzMap(1 << 22, 768, 3840), gq=None, gk=None, at=None, dq=1 << 23, dk=None, work=ws, size=1 << 30, **change):
        return lib.map_qk_norm_grad(nat.RzQk(**{**good, **change}), dy, x, dx, gq, gk, at, dq, dk, work, size, None)

    inf, nan = float("inf"), float("nan")
    for change in (dict(D=31), dict(D=0), dict(D=258, C=600, out_C=600), dict(q_heads=0, k_heads=0), dict(q_heads=-1), dict(k_heads=2),
                   dict(C=63), dict(out_C=63), dict(row_pairs=-1), dict(col_pairs=-1), dict(row_pairs=9), dict(row_pairs=17, col_pairs=0),
                   dict(eps=-1.0), dict(eps=nan), dict(eps=inf), dict(base=0.0), dict(base=-2.0), dict(base=inf), dict(base=nan),
                   dict(scale=inf), dict(scale=nan), dict(dtype=0), dict(dtype=5), dict(N=-1), dict(q_heads=1 << 30),
                   dict(x=None), dict(x=nat.RzMap(1 << 20, 766, 3840)), dict(x=nat.RzMap((1 << 20) + 1, 768, 3840)), dict(gq=2), dict(gk=1), dict(at=4)):
        assert call(**change) == ARG and grad(**change) == ARG, change
    assert call(y=None) == ARG and call(y=nat.RzMap((1 << 20) + 64, 512, 2048)) == ARG
    assert call(y=x) == ARG                       # the same place, but other channels
    many = dict(N=1 << 15, H=1 << 8, W=1 << 8, C=2, out_C=2, q_heads=1, k_heads=0, D=2, row_pairs=0, col_pairs=1)
    assert call(x=nat.RzMap(1 << 40, 1024, 1 << 18), y=nat.RzMap(1 << 50, 1024, 1 << 18), **many) == UNSUPPORTED
    assert lib.map_qk_norm_grad_workspace(nat.RzQk(**good), None) == ARG and lib.map_qk_norm_grad_workspace(None, ctypes.byref(n)) == ARG
    assert lib.map_qk_norm_grad_workspace(nat.RzQk(**good), ctypes.byref(n)) == 0 and n.value >= 4 * 2 * 32
    for change in (dict(dy=None), dict(dx=None), dict(dx=x), dict(dx=nat.RzMap((1 << 21) + 64, 768, 3840)), dict(dq=2), dict(dk=6),
                   dict(work=None), dict(work=ws + 8), dict(size=16)):
        assert grad(**change) == ARG, change
    assert call(N=0, x=None, y=None) == 0 and grad(N=0, dy=None, x=None, dx=None, dq=None, work=None, size=0) == 0


def test_position_bias_refuses(lib, nat):
    good = dict(N=2, heads=3, q_h=2, q_w=3, k_h=4, k_w=2, row_buckets=5, col_buckets=7, dtype=1)
    out, far = nat.RzMap(1 << 20, 32, 192), nat.RzMap(1 << 21, 32, 192)
    t, r, c, n, ws = 1 << 22, 1 << 23, 1 << 24, ctypes.c_size_t(7), 1 << 30

    def call(t=t, r=r, c=c, s=None, out=out, **change):
        return lib.map_position_bias(nat.RzBias(**{**good, **change}), t, r, c, s, out, None)

    def grad(d=out, r=r, c=c, dt=t, work=ws, size=1 << 30, **change):
        return lib.map_position_bias_grad(nat.RzBias(**{**good, **change}), d, r, c, dt, work, size, None)

    for change in (dict(N=-1), dict(heads=0), dict(q_h=-1), dict(k_w=-1), dict(k_h=300, k_w=300), dict(q_h=1 << 16, q_w=2), dict(row_buckets=0),
                   dict(col_buckets=0), dict(row_buckets=1 << 12, col_buckets=(1 << 10) + 1), dict(dtype=0), dict(dtype=4), dict(N=1 << 24),
                   dict(heads=1 << 17), dict(r=None), dict(c=None), dict(r=2), dict(c=1)):
        assert call(**change) == ARG and grad(**change) == ARG, change
    for change in (dict(t=None), dict(t=2), dict(out=None), dict(out=nat.RzMap(1 << 20, 28, 192)), dict(out=nat.RzMap(1 << 20, 32, 188)),
                   dict(out=nat.RzMap((1 << 20) + 2, 32, 192)), dict(s=nat.RzMap((1 << 20) + 32, 32, 192)), dict(s=nat.RzMap(1 << 21, 34, 192))):
        assert call(**change) == ARG, change
    assert lib.map_position_bias_grad_workspace(nat.RzBias(**good), None) == ARG
    assert lib.map_position_bias_grad_workspace(nat.RzBias(**good), ctypes.byref(n)) == 0 and n.value > 0
    for change in (dict(d=None), dict(dt=None), dict(dt=2), dict(work=None), dict(work=ws + 4), dict(size=8), dict(d=nat.RzMap(1 << 20, 28, 192))):
        assert grad(**change) == ARG, change
    assert call(N=0, out=None, t=None, r=None, c=None) == 0
    for change in (dict(q_w=0), dict(k_h=0)):
        assert call(out=None, **change) == 0 and lib.map_position_bias_grad_workspace(nat.RzBias(**{**good, **change}), ctypes.byref(n)) == 0
        assert n.value == 0


def test_position_bias_past_the_grid(lib, nat):
    """A table of more entries than a launch has warps, and more rows and heads than it has blocks."""
    d, n = nat.RzBias(N=1, heads=1 << 13, q_h=1, q_w=1, k_h=1, k_w=1, row_buckets=1 << 11, col_buckets=1 << 11, dtype=1), ctypes.c_size_t(7)
    one = nat.RzMap(1 << 20, 4, 4)
    assert lib.map_position_bias_grad_workspace(d, ctypes.byref(n)) == UNSUPPORTED
    assert lib.map_position_bias_grad(d, one, 1 << 23, 1 << 24, 1 << 22, 1 << 30, 1 << 30, None) == UNSUPPORTED
    d = nat.RzBias(N=1, heads=1 << 16, q_h=1, q_w=1 << 16, k_h=2, k_w=1, row_buckets=1, col_buckets=1, dtype=1)
    assert lib.map_position_bias(d, 1 << 22, 1 << 23, 1 << 24, None, nat.RzMap(1 << 40, 8, 1 << 19), None) == UNSUPPORTED


def test_buckets_match_the_definition(lib):
    import bilinear_image_resize_gb300 as rz
    rng = random.Random(1)
    for _ in range(300):
        q, k, exact = rng.randrange(1, 200), rng.randrange(1, 200), rng.randrange(1, 17)
        side = exact + rng.randrange(0, 17)
        reach, shift = exact + rng.randrange(1, 200), rng.randrange(-50, 50)
        assert np.array_equal(rz.map_position_buckets(q, k, exact, side, reach, shift), tok.buckets(q, k, exact, side, reach, shift))
    # borders that are whole numbers: 8 (128 / 8)^(j / 8) for j = 2, 4, 6
    b = rz.map_position_buckets(1, 200, 8, 16, 128)
    assert [int(b[d]) - 15 for d in (7, 8, 15, 16, 31, 32, 63, 64, 127, 128, 199)] == [7, 8, 9, 10, 11, 12, 13, 14, 15, 15, 15]
    assert np.array_equal(rz.map_position_buckets(65536, 65536, 1, 1024, 65536), rz.map_position_buckets(65536, 65536, 1, 1024, 65536))


def test_buckets_refuse(lib):
    import bilinear_image_resize_gb300 as rz
    out = np.zeros(16, np.int32)
    for bad in ((0, 4, 0, 2, 4, 8), (4, 0, 0, 2, 4, 8), (4, 4, 0, 0, 4, 8), (4, 4, 0, 5, 4, 8), (4, 4, 0, 2, 1025, 8), (4, 4, 0, 2, 4, 2),
                (4, 4, 65537, 2, 4, 8), (4, 4, -65537, 2, 4, 8), (4, 4, 0, 2, 4, 65537), (65537, 4, 0, 2, 4, 8)):
        assert lib.map_position_buckets(*bad, out.ctypes.data) == ARG, bad
    assert lib.map_position_buckets(4, 4, 0, 2, 4, 8, None) == ARG
    for bad in ((0, 4, 2, 4, 8), (4, 1 << 40, 2, 4, 8), (4, 4, 1 << 40, 4, 8), (4, 4, 2, 4, 1 << 33)):
        with pytest.raises(ValueError):
            rz.map_position_buckets(*bad)
    with pytest.raises(rz.ResizeError):
        rz.map_position_buckets(4, 4, 2, 1, 8)


def test_binding_names():
    import bilinear_image_resize_gb300 as rz
    for name in ("map_linear", "map_linear_grad", "map_linear_workspace", "map_linear_grad_workspace", "map_qk_norm", "map_qk_norm_grad",
                 "map_qk_norm_grad_workspace", "map_position_bias", "map_position_bias_grad", "map_position_bias_grad_workspace",
                 "map_position_buckets"):
        assert name in rz.__all__ and getattr(rz, name).__doc__


@pytest.mark.parametrize("pixels, C, K", [(65536, 1024, 4096), (1 << 18, 4096, 4096), (2_200_000, 4096, 4096), (1 << 24, 64, 64), (5000, 1000, 300),
                                          ((1 << 31) - 1, 8, 8), (100, 65536, 65536), (300, 1030, 8)])
@pytest.mark.parametrize("dtype, wtype", [(1, 1), (2, 2), (2, 1), (3, 1)])
def test_workspaces_stay_of_the_size_of_the_maps(lib, nat, pixels, C, K, dtype, wtype):
    """Whatever the sum's length: the operands' layouts (6 bytes an element of float32, 2 of 16 bits, 4 of a dz for a float32 dweight,
    rows rounded to 16 bytes), one float32 matrix of the largest result's size or 64 MB, and a row of sums for every few pixels."""
    es, ws = 4 if dtype == 1 else 2, 4 if wtype == 1 else 2
    d = nat.RzLinear(1, 1, pixels, C, K, dtype, 1)
    at = [1 << 48, 1 << 49, 1 << 50, 1 << 51, 1 << 52, 1 << 53]
    x, y, pre, dx = (nat.RzMap(a, pixels * n * es, pixels * n * es) for a, n in zip(at, (C, K, K, C)))
    n = ctypes.c_size_t(0)
    up = lambda v: (v + 7) // 8 * 8       # noqa: E731
    laid = 6 if dtype == 1 else 2
    most = 64 << 20
    assert lib.map_linear_workspace(d, x, at[4], C * es, None, None, y, ctypes.byref(n)) == 0
    assert n.value <= laid * up(C) * (pixels + K) + max(4 * pixels * up(K), most) + 1024
    assert lib.map_linear_grad_workspace(d, y, x, at[4], C * es, pre, dx, at[5], C * ws, wtype, ctypes.byref(n)) == 0
    operands = laid * (up(C) * (pixels + K)) + (4 if (dtype, wtype) in ((2, 1), (3, 1)) else laid) * up(K) * pixels
    assert n.value <= operands + max(4 * pixels * up(C), 4 * K * up(C), most) + 4 * K * 700 + 4096
    # towards the weight alone
    assert lib.map_linear_grad_workspace(d, y, x, at[4], C * es, pre, None, at[5], C * ws, wtype, ctypes.byref(n)) == 0
    assert n.value <= operands + max(4 * K * up(C), most) + 4 * K * 700 + 4096
