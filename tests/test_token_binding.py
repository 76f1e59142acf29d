"""What the binding of the operators around attention hands to the library, and
what it refuses before any call.  The tensors are stand-ins without memory and
the library's functions are recorders with the binding's own ctypes signatures,
so nothing is launched and no GPU is needed."""
import pytest

torch = pytest.importorskip("torch")

from test_map_binding import Standin, calls, rz, standins    # noqa: E402,F401

F32, BF16, INT = torch.float32, torch.bfloat16, torch.int32


def every_call(rz):                                           # noqa: F811
    """name -> (a call of the operator with the given tensors, their shapes and types): all that an entry takes."""
    x, y, w, b = ((2, 4, 4, 16), BF16), ((2, 4, 4, 24), BF16), ((24, 16), BF16), ((24,), F32)
    qkv, qk, g, at = ((2, 4, 4, 96), BF16), ((2, 4, 4, 64), BF16), ((32,), F32), ((2, 4, 4, 2), INT)
    table, rows, cols, s = ((5, 7, 3), F32), ((5,), INT), ((4,), INT), ((2, 3, 6, 8), BF16)
    grids = dict(query=(2, 3), key=(4, 2))
    return {
        "linear": (lambda **t: rz.map_linear(act=2, stream=0, **t), dict(x=x, y=y, weight=w, bias=b, residual=y, pre=y)),
        "linear_grad": (lambda **t: rz.map_linear_grad(act=2, stream=0, **t),
                        dict(dy=y, x=x, weight=w, dx=x, dweight=w, dbias=b, pre=y)),
        "qk": (lambda **t: rz.map_qk_norm(q_heads=1, k_heads=1, head_dim=32, stream=0, **t),
               dict(x=qkv, y=qk, gamma_q=g, gamma_k=g, positions=at)),
        "qk_grad": (lambda **t: rz.map_qk_norm_grad(q_heads=1, k_heads=1, head_dim=32, stream=0, **t),
                    dict(dy=qk, x=qkv, dx=qkv, gamma_q=g, gamma_k=g, dgamma_q=g, dgamma_k=g, positions=at)),
        "bias": (lambda **t: rz.map_position_bias(stream=0, **grids, **t), dict(table=table, rows=rows, cols=cols, out=s, scores=s)),
        "bias_grad": (lambda **t: rz.map_position_bias_grad(stream=0, **grids, **t), dict(dout=s, rows=rows, cols=cols, dtable=table)),
    }


OPS = ["linear", "linear_grad", "qk", "qk_grad", "bias", "bias_grad"]
LAUNCHES = ("map_linear", "map_linear_grad", "map_qk_norm", "map_qk_norm_grad", "map_position_bias", "map_position_bias_grad")


def strided(spec, name, strides):
    t = standins(spec)
    shape, dtype = spec[name]
    t[name] = Standin(shape, dtype, at=1 << 50, strides=strides)
    return t


@pytest.mark.parametrize("op", OPS)
def test_tensors_of_another_device_are_refused(rz, calls, op):    # noqa: F811
    call, spec = every_call(rz)[op]
    for name in spec:
        for t in (standins(spec, name, device=1), standins(spec, name, cuda=False)):
            with pytest.raises(ValueError):
                call(**t)
    with pytest.raises(ValueError):
        call(**standins(spec, home=1))
    assert not any(n in LAUNCHES for n, _ in calls)
    call(**standins(spec))
    assert any(n in LAUNCHES for n, _ in calls)


@pytest.mark.parametrize("op", OPS)
def test_other_types_and_shapes_are_refused(rz, calls, op):       # noqa: F811
    call, spec = every_call(rz)[op]
    for name, (shape, dtype) in spec.items():
        wrong = [torch.float64, torch.int64 if dtype is INT else torch.float16 if dtype is BF16 else torch.float64]
        if name in ("dweight",):
            wrong = [torch.float64, torch.float16]
        for other in wrong:
            if name in ("x", "out", "dout") and other is torch.float16 and len(spec) == 0:
                continue
            t = standins(spec)
            t[name] = Standin(shape, other, at=1 << 50)
            if name == "dweight" and other is torch.float16:
                continue                                      # the library's to refuse
            if name == "dout" and other is torch.float16:
                continue                                      # dout alone has that type: taken
            with pytest.raises(ValueError):
                call(**t)
        for bad in ((*shape[:-1], shape[-1] + 1), (*shape, 1, 1)):
            if op.startswith("qk") and name in ("x", "y", "dy") and len(bad) == len(shape):
                continue                                      # more channels than the heads' are taken
            t = standins(spec)
            t[name] = Standin(bad, dtype, at=1 << 50)
            with pytest.raises(ValueError):
                call(**t)
    assert not any(n in LAUNCHES for n, _ in calls)


def test_layouts_that_are_refused(rz, calls):                     # noqa: F811
    every = every_call(rz)
    for op, name, strides in (("linear", "weight", (1, 24)), ("linear", "weight", (8, 1)), ("linear", "x", (256, 64, 32, 1)),
                              ("linear_grad", "dweight", (16, 2)), ("qk", "positions", (64, 16, 4, 1)), ("qk", "gamma_q", (2,)),
                              ("bias", "out", (1, 8, 6, 1)), ("bias", "out", (144, 48, 8, 2)), ("bias", "rows", (2,)),
                              ("bias", "table", (1, 5, 35)), ("bias", "scores", (200, 48, 8, 1))):
        call, spec = every[op]
        with pytest.raises(ValueError):
            call(**strided(spec, name, strides))
    assert not any(n in LAUNCHES for n, _ in calls)


def test_padded_weights_and_matrices(rz, calls):                  # noqa: F811
    every = every_call(rz)
    call, spec = every["linear"]
    call(**strided(spec, "weight", (40, 1)))
    assert calls[-1][0] == "map_linear" and calls[-1][1][2:4] == (1 << 50, 80)
    t = Standin((2, 3, 6, 8), BF16, at=1 << 50, strides=(270, 90, 15, 1))
    n, m = rz._matrices(t, "out", 3, 6, 8)
    assert (n, m.data, m.pitch, m.batch_stride) == (2, 1 << 50, 30, 180)
    n, m = rz._matrices(Standin((4, 1, 6, 8), BF16, at=1 << 50, strides=(90, 7, 15, 1)), "out", 1, 6, 8)
    assert (n, m.pitch, m.batch_stride) == (4, 30, 180)       # one head: the batch's own stride
    call, spec = every["bias"]
    call(**{**standins(spec), "out": t})
    assert calls[-1][0] == "map_position_bias"


@pytest.mark.parametrize("op", ["linear", "linear_grad", "qk_grad", "bias_grad"])
def test_workspaces_that_are_not_the_calls_own_memory_are_refused(rz, calls, op):   # noqa: F811
    call, spec = every_call(rz)[op]
    u8, n = torch.uint8, 1 << 20
    for bad in (Standin((n,), u8, cuda=False), Standin((n,), u8, device=1), Standin((n,), u8, strides=(0,)), Standin((n // 2,), u8, strides=(2,))):
        with pytest.raises(ValueError):
            call(**standins(spec), workspace=bad)
    assert not calls
    call(**standins(spec), workspace=Standin((n // 4,), F32, at=1 << 50))
    (name, got), = calls
    assert name in LAUNCHES and (1 << 50) in got and n in got


@pytest.mark.parametrize("op", ["linear", "linear_grad"])
def test_status_words(rz, calls, op):                             # noqa: F811
    call, spec = every_call(rz)[op]
    for bad in (Standin((1,), torch.int64), Standin((2,), INT), Standin((1,), INT, device=1), Standin((1,), INT, cuda=False)):
        with pytest.raises(ValueError):
            call(**standins(spec), status=bad)
    call(**standins(spec), status=Standin((1,), INT, at=1 << 51))
    assert (1 << 51) in calls[-1][1]


def test_sizes_past_an_int_are_refused(rz, calls):                # noqa: F811
    big = 1 << 32
    x, y = Standin((1, 1, 1, 16)), Standin((1, 1, 1, big))
    with pytest.raises(ValueError):
        rz.map_linear(x, y, Standin((big, 16)), stream=0)
    q = Standin((1, 1, 1, 64))
    for bad in (dict(q_heads=big + 1), dict(k_heads=big + 1), dict(head_dim=big + 32), dict(row_pairs=big, col_pairs=0), dict(col_pairs=big)):
        with pytest.raises(ValueError):
            rz.map_qk_norm(q, Standin((1, 1, 1, 64), at=1 << 45), **{**dict(q_heads=1, k_heads=1, head_dim=32), **bad}, stream=0)
    t, i, s = Standin((3, 3, 2), F32), Standin((3,), INT), Standin((1, 2, 4, 4))
    for bad in (((big + 2, 2), (2, 2)), ((2, 2), (2, big + 2))):
        with pytest.raises(ValueError):
            rz.map_position_bias(t, i, i, s, *bad, stream=0)
    with pytest.raises(ValueError):
        rz.map_linear(x, Standin((1, 1, 1, 16), at=1 << 45), Standin((16, 16)), act=big + 1, stream=0)
    assert not calls


def test_few_pixels_ask_for_no_workspace(rz, calls):              # noqa: F811
    rz.map_linear(Standin((8, 1, 1, 16)), Standin((8, 1, 1, 16), at=1 << 45), Standin((16, 16), at=1 << 46), stream=0)
    (name, got), = calls
    assert name == "map_linear" and got[8:10] == (None, 0)


@pytest.mark.parametrize("op", ["linear", "linear_grad"])
def test_a_time_out_of_an_earlier_call_is_raised(rz, calls, monkeypatch, op):    # noqa: F811
    """Without a status word of the caller's, calls hand on the binding's own one of the device."""
    import ctypes
    from bilinear_image_resize_gb300 import _native
    call, spec = every_call(rz)[op]
    word = ctypes.c_int(0)
    monkeypatch.setitem(rz._waits, 0, (word, ctypes.addressof(word), word))
    monkeypatch.setattr(_native.load(), "resize_strerror", lambda code: b"timeout", raising=False)
    call(**standins(spec))
    assert ctypes.addressof(word) in calls[-1][1]
    word.value = rz.RZ_ERR_TIMEOUT                            # as a kernel leaves it
    before = len([n for n, _ in calls if n in LAUNCHES])
    with pytest.raises(rz.ResizeError, match="earlier") as e:
        call(**standins(spec))
    assert e.value.code == rz.RZ_ERR_TIMEOUT and word.value == 0
    assert len([n for n, _ in calls if n in LAUNCHES]) == before
    call(**standins(spec))                                    # told once
    word.value = rz.RZ_ERR_TIMEOUT
    call(**standins(spec), status=Standin((1,), INT, at=1 << 51))     # the caller's own word: theirs to look at
    assert (1 << 51) in calls[-1][1] and word.value == rz.RZ_ERR_TIMEOUT
