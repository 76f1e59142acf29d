"""Host-side checks of the feature-map entry points: arguments refused before
any CUDA call, struct layouts, workspace sizes.  No GPU needed."""
import ctypes
import os

import pytest

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


@pytest.mark.parametrize("cname, pyname", [("rz_map", "RzMap"), ("rz_drop", "RzDrop"), ("rz_norm", "RzNorm"),
                                           ("rz_resample", "RzResample")])
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


def test_group_norm_refuses(lib, nat):
    good = dict(N=2, H=4, W=4, C=12, groups=3, dtype=1, act=1, eps=1e-5)
    n = ctypes.c_size_t(7)

    def query(**change):
        return lib.map_group_norm_workspace(nat.RzNorm(**{**good, **change}), ctypes.byref(n))

    assert query() == 0 and n.value > 0
    assert lib.map_group_norm_workspace(None, ctypes.byref(n)) == ARG
    assert lib.map_group_norm_workspace(nat.RzNorm(**good), None) == ARG
    for change in (dict(N=-1), dict(H=-1), dict(W=-2), dict(C=0), dict(C=65537, groups=1), dict(groups=0), dict(groups=5),
                   dict(dtype=0), dict(dtype=4), dict(act=-1), dict(act=3), dict(eps=0.0), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(eps=float("inf")), dict(H=1 << 16, W=1 << 15)):
        assert query(**change) == ARG, change
    assert query(N=65536) == UNSUPPORTED
    assert query(N=0) == 0 and n.value == 0
    d, m = nat.RzNorm(**good), nat.RzMap(1 << 20, 192, 768)
    far, ws = nat.RzMap(1 << 21, 192, 768), 1 << 30

    def norm(x=m, y=far, drop=None, gamma=None, mean=None, w=ws, size=1 << 20):
        return lib.map_group_norm(d, drop, x, y, gamma, None, mean, None, w, size, None)

    assert norm(x=None) == ARG and norm(y=None) == ARG
    assert norm(y=m) == ARG and norm(y=nat.RzMap((1 << 20) + 1000, 192, 768)) == ARG      # overlapping
    assert norm(x=nat.RzMap((1 << 20) + 2, 192, 768)) == ARG                              # not an element's alignment
    assert norm(x=nat.RzMap(1 << 20, 188, 768)) == ARG and norm(x=nat.RzMap(1 << 20, 192, 764)) == ARG
    assert norm(x=nat.RzMap(1 << 20, 194, 800)) == ARG
    assert norm(gamma=2) == ARG and norm(mean=6) == ARG
    assert norm(drop=nat.RzDrop(-0.1, 0, 0)) == ARG and norm(drop=nat.RzDrop(1.5, 0, 0)) == ARG
    assert norm(drop=nat.RzDrop(float("nan"), 0, 0)) == ARG
    assert norm(w=None) == ARG and norm(w=ws + 8) == ARG and norm(size=16) == ARG
    args = (None, None, 1 << 22, 1 << 23, None, None, ws, 1 << 20, None)
    assert lib.map_group_norm_grad(d, None, m, m, far, None, None, None, 1 << 23, None, None, ws, 1 << 20, None) == ARG
    assert lib.map_group_norm_grad(d, None, m, far, far, *args) == ARG
    assert lib.map_group_norm_grad(d, None, far, m, far, *args) == ARG
    assert lib.map_group_norm_grad(d, None, m, m, None, *args) == ARG
    empty = nat.RzNorm(**{**good, "N": 0})
    assert lib.map_group_norm(empty, None, None, None, None, None, None, None, None, 0, None) == 0


def test_dropout_refuses(lib, nat):
    m, far, d = nat.RzMap(1 << 20, 64, 256), nat.RzMap(1 << 21, 64, 256), nat.RzDrop(0.1, 1, 2)

    def drop(x=m, r=None, y=far, n=2, h=4, w=4, c=4, dtype=1, spec=d):
        return lib.map_dropout(x, r, y, n, h, w, c, dtype, spec, None)

    for bad in (dict(x=None), dict(y=None), dict(spec=None), dict(spec=nat.RzDrop(2.0, 0, 0)), dict(dtype=0), dict(c=0),
                dict(n=-1), dict(y=nat.RzMap((1 << 20) + 64, 64, 256)), dict(r=nat.RzMap((1 << 21) + 64, 64, 256)),
                dict(x=nat.RzMap(1 << 20, 60, 256)), dict(y=nat.RzMap((1 << 21) + 1, 64, 256)),
                dict(y=nat.RzMap(1 << 20, 64, 260))):
        assert drop(**bad) == ARG, bad
    assert drop(x=None, y=None, n=0) == 0 and drop(x=None, y=None, h=0) == 0


def test_resize_map_refuses(lib, nat):
    good = dict(N=2, src_n=2, H=4, W=4, out_h=6, out_w=6, C=4, dtype=1, src_dtype=1)
    src, dst = nat.RzMap(1 << 20, 64, 256), nat.RzMap(1 << 21, 96, 576)
    n = ctypes.c_size_t(7)

    def fwd(s=src, b=None, o=dst, **change):
        return lib.resize_map(nat.RzResample(**{**good, **change}), s, b, o, None)

    assert lib.resize_map(None, src, None, dst, None) == ARG
    for change in (dict(src_n=3), dict(src_n=0), dict(H=0), dict(W=0), dict(H=65537), dict(out_h=-1), dict(out_w=65537),
                   dict(C=0), dict(dtype=0), dict(dtype=2, src_dtype=3), dict(dtype=1, src_dtype=2)):
        assert fwd(**change) == ARG, change
    assert fwd(N=70000, src_n=70000) == UNSUPPORTED
    assert fwd(s=None) == ARG and fwd(o=None) == ARG
    assert fwd(o=nat.RzMap((1 << 20) + 128, 96, 576)) == ARG
    assert fwd(b=nat.RzMap((1 << 21) + 96, 96, 576)) == ARG
    assert fwd(s=nat.RzMap(1 << 20, 60, 256)) == ARG and fwd(o=nat.RzMap(1 << 21, 96, 500)) == ARG
    assert fwd(out_h=0, s=None, o=None) == 0
    d = nat.RzResample(**{**good, "src_n": 1})
    assert lib.resize_map_grad_workspace(d, ctypes.byref(n)) == 0 and n.value == 4 * 6 * 6 * 4
    assert lib.resize_map_grad_workspace(nat.RzResample(**good), ctypes.byref(n)) == 0 and n.value == 0
    assert lib.resize_map_grad_workspace(d, None) == ARG
    assert lib.resize_map_grad(d, dst, src, None, 0, None) == ARG
    assert lib.resize_map_grad(d, dst, src, 1 << 30, 100, None) == ARG
    assert lib.resize_map_grad(d, dst, src, (1 << 30) + 4, 1 << 20, None) == ARG
    assert lib.resize_map_grad(nat.RzResample(**good), dst, nat.RzMap((1 << 21) + 64, 64, 256), None, 0, None) == ARG
    assert lib.resize_map_grad(nat.RzResample(**good), None, src, None, 0, None) == ARG


def test_binding_names():
    import bilinear_image_resize_gb300 as rz
    for name in ("map_group_norm", "map_group_norm_grad", "map_group_norm_workspace", "map_dropout", "resize_map",
                 "resize_map_grad", "resize_map_grad_workspace"):
        assert name in rz.__all__ and getattr(rz, name).__doc__
