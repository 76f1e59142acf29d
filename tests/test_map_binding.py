"""What the binding of the feature-map operators hands to the library: sizes
past 32 bits, and what it refuses before any call.  The tensors are stand-ins
without memory and the library's functions are recorders with the binding's
own ctypes signatures, so nothing is launched and no GPU is needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


class Standin:
    """A CUDA tensor's shape, strides and type over no memory."""

    def __init__(self, shape, dtype=torch.bfloat16, device=0, at=1 << 40, strides=None, cuda=True):
        self.meta = torch.empty(shape, dtype=dtype, device="meta")
        if strides:
            self.meta = self.meta.as_strided(shape, strides)
        self.dtype, self.shape, self.is_cuda, self.index, self.at = dtype, self.meta.shape, cuda, device, at
        self.device = torch.device("cuda", device) if cuda else torch.device("cpu")

    def data_ptr(self):
        return self.at

    def get_device(self):
        return self.index if self.is_cuda else -1

    def __getattr__(self, name):
        return getattr(self.meta, name)


@pytest.fixture
def rz():
    import bilinear_image_resize_gb300 as m
    return m


@pytest.fixture
def calls(rz, monkeypatch):
    """(name, arguments as the library would receive them) of every call."""
    from bilinear_image_resize_gb300 import _native
    made, kept = [], []

    class Library:
        pass

    def recorder(name, res, args):
        def record(*got):
            made.append((name, got))
            return 0
        return ctypes.CFUNCTYPE(res, *args)(record)

    lib = Library()
    for name, (res, args) in _native.SIGNATURES.items():
        if name.startswith(("map_", "resize_map")):
            f = recorder(name, res, args)
            kept.append(f)
            setattr(lib, name, f)
    monkeypatch.setattr(_native, "load", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return made


LARGE = [(1 << 32,), (1, 1 << 32), (1 << 32, 1), (64, 8192, 8192, 1), ((1 << 32) + 5,), ((1 << 32) + 5, 1), (1 << 31,),
         ((1 << 31) + 11,), (3, (1 << 31) + 11), (1 << 16, 1 << 16, 3)]


@pytest.mark.parametrize("shape", LARGE + [(7,), (), (3, 0), (2, 3, 5, 4, 2)])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_takes_every_element_of_packed_tensors(rz, calls, shape, residual):
    x, y, r = Standin(shape), Standin(shape, at=1 << 41), Standin(shape, at=1 << 42) if residual else None
    rz.map_dropout(x, y, 0.5, 1, residual=r, stream=0)
    done = 0
    for name, a in calls:
        if name == "map_dropout_packed":
            assert (a[0], a[1], a[2], a[4]) == (1 << 40, (1 << 42) if residual else None, 1 << 41, 2)
            done += a[3]
        else:
            n, h, w, c = a[3:7]
            assert name == "map_dropout" and min(n, h, w, c) >= 0
            done += n * h * w * c
    assert done == x.numel()


# every size of a map past an int, and one that an int would hold as a small number
PAST = [((1 << 32) + 2, 1, 1, 8), (1, (1 << 32) + 2, 1, 8), (1, 1, (1 << 32) + 2, 8), (1, 1, 1, (1 << 32) + 8),
        (1, 1, 1 << 32, 8), (1 << 31, 1, 1, 8), (1, 1 << 31, 1, 8)]


@pytest.mark.parametrize("shape", PAST)
def test_sizes_past_an_int_are_refused(rz, calls, shape):
    x, y = Standin(shape), Standin(shape, at=1 << 50)
    small, g = Standin((1, 2, 2, shape[3])), Standin((shape[0], 2), torch.float32)
    for call in (lambda: rz.map_group_norm(x, y, 2, stream=0), lambda: rz.map_group_norm_workspace(x, 2),
                 lambda: rz.map_group_norm_grad(x, x, y, 2, mean=g, rstd=g, stream=0),
                 lambda: rz.resize_map(x, y, stream=0), lambda: rz.resize_map(small, y, stream=0),
                 lambda: rz.resize_map_grad(x, y, stream=0), lambda: rz.resize_map_grad(y, small, stream=0),
                 lambda: rz.resize_map_grad_workspace(x, y)):
        with pytest.raises(ValueError):
            call()
    assert not calls


def test_strided_sizes_past_an_int_are_refused_by_dropout(rz, calls):
    shape, strides = (2, 1 << 32, 1, 8), (16 << 32, 16, 8, 1)
    with pytest.raises(ValueError):
        rz.map_dropout(Standin(shape, strides=strides), Standin(shape, strides=strides, at=1 << 50), 0.5, 1, stream=0)
    assert not calls


@pytest.mark.parametrize("change", [dict(groups=(1 << 32) + 2), dict(groups=-(1 << 32) + 2), dict(act=(1 << 32) + 1)])
def test_groups_and_activation_past_an_int_are_refused(rz, calls, change):
    x, y, m = Standin((2, 4, 4, 8)), Standin((2, 4, 4, 8), at=1 << 50), Standin((2, 2), torch.float32)
    kw = {**dict(groups=2, act=0), **change}
    stats = {} if "groups" in change else dict(mean=m, rstd=m)
    for call in (lambda: rz.map_group_norm(x, y, stream=0, **kw),
                 lambda: rz.map_group_norm_grad(x, x, y, stream=0, **stats, **kw)):
        with pytest.raises(ValueError):
            call()
    if "groups" in change:
        with pytest.raises(ValueError):
            rz.map_group_norm_workspace(x, kw["groups"])
    assert not calls


def every_call(rz):
    """name -> (a call of the operator with the given tensors, their names, shapes and types): all that an entry takes."""
    f32, bf16 = torch.float32, torch.bfloat16
    x = ((2, 4, 4, 8), bf16)
    c, s = ((8,), f32), ((2, 2), f32)
    norm = dict(x=x, y=x, gamma=c, beta=c, mean=s, rstd=s)
    grad = dict(dy=x, x=x, dx=x, gamma=c, beta=c, mean=s, rstd=s, dgamma=c, dbeta=c)
    return {
        "dropout": (lambda x, y, residual: rz.map_dropout(x, y, 0.5, 1, residual=residual, stream=0),
                    dict(x=x, y=x, residual=x)),
        "norm": (lambda **t: rz.map_group_norm(groups=2, stream=0, **t), norm),
        "norm_grad": (lambda **t: rz.map_group_norm_grad(groups=2, stream=0, **t), grad),
        "resize": (lambda **t: rz.resize_map(stream=0, **t), dict(src=((2, 2, 2, 8), bf16), dst=x, base=x)),
        "resize_grad": (lambda **t: rz.resize_map_grad(stream=0, **t), dict(ddst=x, dsrc=((1, 2, 2, 8), f32))),
    }


def standins(spec, strange=None, device=0, cuda=True, home=0):
    return {k: Standin(shape, dtype, at=(64 + i) << 40, device=device if k == strange else home, cuda=cuda or k != strange)
            for i, (k, (shape, dtype)) in enumerate(spec.items())}


@pytest.mark.parametrize("op", ["dropout", "norm", "norm_grad", "resize", "resize_grad"])
def test_tensors_of_another_device_are_refused(rz, calls, op):
    call, spec = every_call(rz)[op]
    for name in spec:
        for t in (standins(spec, name, device=1), standins(spec, name, cuda=False)):
            with pytest.raises(ValueError):
                call(**t)
    # all of them on one that is not current
    with pytest.raises(ValueError):
        call(**standins(spec, home=1))
    assert not any(n in ("map_dropout", "map_dropout_packed", "map_group_norm", "map_group_norm_grad", "resize_map",
                         "resize_map_grad") for n, _ in calls)
    call(**standins(spec))
    assert calls


@pytest.mark.parametrize("op", ["norm", "norm_grad", "resize_grad"])
def test_workspaces_that_are_not_the_calls_own_memory_are_refused(rz, calls, op):
    call, spec = every_call(rz)[op]
    u8, n = torch.uint8, 1 << 20
    # host memory, another device's, one byte seen n times, every other byte
    for bad in (Standin((n,), u8, cuda=False), Standin((n,), u8, device=1), Standin((n,), u8, strides=(0,)),
                Standin((n // 2,), u8, strides=(2,))):
        with pytest.raises(ValueError):
            call(**standins(spec), workspace=bad)
    assert not calls
    call(**standins(spec), workspace=Standin((n // 4,), torch.float32, at=1 << 50))
    (name, got), = calls
    assert name in ("map_group_norm", "map_group_norm_grad", "resize_map_grad") and got[-3:] == (1 << 50, n, None)


def test_packed_dropout_refuses():
    from bilinear_image_resize_gb300 import _build, _native
    _build.build()
    lib, d, arg = _native.load(), _native.RzDrop(0.1, 1, 2), 1
    x, y, r = 1 << 20, 1 << 21, 1 << 22

    def drop(x=x, r=None, y=y, n=256, dtype=1, spec=d):
        return lib.map_dropout_packed(x, r, y, n, dtype, spec, None)

    for bad in (dict(x=None), dict(y=None), dict(x=x + 2), dict(y=y + 1), dict(r=r + 2), dict(dtype=0), dict(dtype=4),
                dict(spec=None), dict(spec=_native.RzDrop(-0.1, 0, 0)), dict(spec=_native.RzDrop(float("nan"), 0, 0)),
                dict(n=(1 << 46) + 1), dict(y=x + 1020), dict(x=y + 1020), dict(r=y + 4), dict(r=y - 4)):
        assert drop(**bad) == arg, bad
    # an element at a time, more than the grid's width of blocks
    assert drop(n=1 << 42, x=(1 << 50) + 4, y=(1 << 51) + 4) == 2
    assert drop(x=None, y=None, n=0) == 0


def test_norm_refuses_more_statistics_than_an_int_counts():
    from bilinear_image_resize_gb300 import _build, _native
    _build.build()
    lib, n, unsupported = _native.load(), ctypes.c_size_t(0), 2
    for N, C, groups in ((65535, 65536, 65536), (32768, 65536, 65536), (65535, 65536, 32768)):
        d, m = _native.RzNorm(N, 1, 1, C, groups, 2, 0, 1e-5), _native.RzMap(1 << 40, 2 * C, 2 * C)
        far, want = _native.RzMap(1 << 41, 2 * C, 2 * C), unsupported if N * groups > 0x7fffffff else 0
        assert lib.map_group_norm_workspace(d, ctypes.byref(n)) == want
        # no workspace: refused in any case
        assert lib.map_group_norm(d, None, m, far, None, None, None, None, None, 0, None) == (want or 1)
        assert lib.map_group_norm_grad(d, None, m, m, far, None, None, 1 << 42, 1 << 43, None, None, None, 0,
                                       None) == (want or 1)
    # the most that is taken: 2^31 - 2^16 statistics
    d = _native.RzNorm(32767, 1, 1, 65536, 65536, 2, 0, 1e-5)
    assert lib.map_group_norm_workspace(d, ctypes.byref(n)) == 0 and n.value > 8 * 32767 * 65536


def test_maps_whose_bytes_pass_64_bits_are_refused():
    from bilinear_image_resize_gb300 import _build, _native
    _build.build()
    lib, d, arg = _native.load(), _native.RzDrop(0.1, 1, 2), 1
    top = 1 << 46
    # rows 2^46 bytes apart, 2^18 of them below the last: 2^64, which 64 bits hold as 0
    tall = _native.RzMap(1 << 20, top, 16)
    assert lib.map_dropout(tall, None, tall, 2, (1 << 18) + 1, 1, 4, 1, d, None) == arg
    assert lib.map_dropout(tall, None, tall, 1, (1 << 18) + 1, 1, 4, 1, d, None) == arg
    assert lib.map_dropout(_native.RzMap(1 << 20, top, 16), None, _native.RzMap((1 << 20) + 16, top, 16), 1,
                           (1 << 18) + 1, 1, 4, 1, d, None) == arg
    many = _native.RzMap(1 << 20, 16, top)
    assert lib.map_dropout(many, None, many, (1 << 18) + 1, 1, 1, 4, 1, d, None) == arg
    far = _native.RzMap(1 << 40, 16, 16 * ((1 << 18) + 1))
    r = _native.RzResample(1, 1, 16385, 1, 16385, 1, 4, 1, 1)
    assert lib.resize_map(r, _native.RzMap(1 << 20, top, 0), None, far, None) == arg
