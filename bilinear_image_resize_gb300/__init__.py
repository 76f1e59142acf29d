"""GB300-native image resize: Python binding of the C ABI (include/gbresize.h).

Every function here only marshals arguments (torch tensors -> device pointers,
byte pitches, the current CUDA stream) and calls the C entry point of the
same name; all computation runs in the library's CUDA kernels.  A non-zero
status raises ``ResizeError``.

Images are torch tensors laid out HWC (or HW for one channel) with the last
two dimensions packed; the row pitch is taken from ``stride(0)``, so row
padding (a view into a wider buffer) is allowed.
"""
from __future__ import annotations

import ctypes

from . import _native
from ._native import (KIND_F32, KIND_FILTER3X3, KIND_NORMALIZE, KIND_U8, RZ_BORDER_CLAMP, RZ_BORDER_MIRROR,
                      RZ_BORDER_WRAP, RZ_EPI_FILTER, RZ_EPI_FILTER3X3, RZ_EPI_GRAY_BGR, RZ_EPI_GRAY_RGB, RZ_EPI_NORMALIZE_NCHW, RZ_ERR_ARG, RZ_ERR_CUDA, RZ_ERR_NOMEM, RZ_ERR_TIMEOUT,
                      RZ_ERR_UNSUPPORTED, RZ_F32, RZ_LINEAR, RZ_MAX_DIM, RZ_NEAREST, RZ_NOALLOC_MAX_DIM, RZ_OK,
                      RZ_OPT_CTAS_PER_SM, RZ_OPT_GENERIC_ONLY, RZ_OPT_GRID_MODE, RZ_OPT_PDL, RZ_OPT_RING_ROWS,
                      RZ_MULTI_MAX_JOBS, RZ_OPT_F32_KERNEL, RZ_OPT_FILTER_KERNEL, RZ_OPT_L2_PREFETCH, RZ_COPY_PDL, RZ_COPY_L2_PREFETCH, RZ_FILTER_AUTO, RZ_FILTER_FP32, RZ_FILTER_TENSOR, RZ_OPT_STAGES, RZ_OPT_U8_KERNEL, RZ_U8,
                      RZ_ACT_GELU, RZ_ACT_NONE, RZ_ACT_SILU, RZ_BF16, RZ_F16, RzDrop, RzEpilogue, RzJob, RzMap, RzNorm,
                      RzResample)

__all__ = [
    "ResizeError", "Plan", "resize_plan_create", "resize_plan_destroy", "resize_plan_status",
    "resize_plan_set_tile", "resize_plan_set_option", "resize_u8", "resize_f32", "resize_u8_batch",
    "resize_f32_batch", "resize_fused", "resize_u8_host", "resize_wait_selftest",
    "resize_axis_table", "resize_strerror", "resize_last_cuda_error", "make_epilogue", "resize_u8_noalloc",
    "RZ_NOALLOC_MAX_DIM",
    "RZ_LINEAR", "RZ_NEAREST", "RZ_U8", "RZ_F32", "RZ_EPI_NORMALIZE_NCHW", "RZ_EPI_FILTER3X3",
    "RZ_EPI_GRAY_RGB", "RZ_EPI_GRAY_BGR", "RZ_BORDER_CLAMP", "RZ_BORDER_MIRROR", "RZ_BORDER_WRAP",
    "resize_plan_create_border", "resize_axis_table_border", "RZ_EPI_FILTER", "RZ_OPT_FILTER_KERNEL", "RZ_OPT_F32_KERNEL",
    "filter2d_valid_f32", "Texture", "resize_texture_create", "make_jobs", "resize_u8_multi",
    "RZ_MULTI_MAX_JOBS",
    "RZ_OK", "RZ_ERR_ARG", "RZ_ERR_UNSUPPORTED", "RZ_ERR_CUDA", "RZ_ERR_NOMEM", "RZ_ERR_TIMEOUT",
    "RZ_MAX_DIM", "KIND_U8", "KIND_F32", "KIND_NORMALIZE", "KIND_FILTER3X3",
    "RZ_OPT_STAGES", "RZ_OPT_GENERIC_ONLY", "RZ_OPT_CTAS_PER_SM", "RZ_OPT_GRID_MODE", "RZ_OPT_PDL",
    "RZ_OPT_RING_ROWS", "RZ_OPT_U8_KERNEL", "RZ_OPT_L2_PREFETCH",
    "resize_copy_baseline", "RZ_COPY_PDL", "RZ_COPY_L2_PREFETCH",
    "RZ_FILTER_AUTO", "RZ_FILTER_FP32", "RZ_FILTER_TENSOR",
    "map_group_norm", "map_group_norm_grad", "map_group_norm_workspace", "map_dropout",
    "resize_map", "resize_map_grad", "resize_map_grad_workspace",
    "RZ_BF16", "RZ_F16", "RZ_ACT_NONE", "RZ_ACT_SILU", "RZ_ACT_GELU",
]


class ResizeError(RuntimeError):
    def __init__(self, code: int, where: str):
        lib = _native.load()
        msg = lib.resize_strerror(code).decode()
        if code == RZ_ERR_CUDA:
            msg += f" (cudaError {lib.resize_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [status {code}]")
        self.code = code


def _check(code: int, where: str) -> None:
    if code != RZ_OK:
        raise ResizeError(code, where)


def _stream(stream) -> int:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owns an ``rz_plan`` handle; freed by ``resize_plan_destroy`` or on collection."""

    def __init__(self, handle: int, in_h: int, in_w: int, out_h: int, out_w: int, mode: int,
                 border: int = RZ_BORDER_CLAMP):
        self.handle = handle
        self.in_h, self.in_w, self.out_h, self.out_w, self.mode = in_h, in_w, out_h, out_w, mode
        self.border = border

    def destroy(self) -> None:
        if self.handle:
            h, self.handle = self.handle, None
            _check(_native.load().resize_plan_destroy(h), "resize_plan_destroy")

    def __del__(self):
        try:
            if self.handle:
                _native.load().resize_plan_destroy(self.handle)
                self.handle = None
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def resize_plan_create(in_h: int, in_w: int, out_h: int, out_w: int, mode: int = RZ_LINEAR, stream=None,
                       border: int = RZ_BORDER_CLAMP) -> Plan:
    if border != RZ_BORDER_CLAMP:
        return resize_plan_create_border(in_h, in_w, out_h, out_w, mode, border, stream)
    h = ctypes.c_void_p()
    _check(_native.load().resize_plan_create(ctypes.byref(h), in_h, in_w, out_h, out_w, mode, _stream(stream)),
           "resize_plan_create")
    return Plan(h.value, in_h, in_w, out_h, out_w, mode)


def resize_plan_create_border(in_h: int, in_w: int, out_h: int, out_w: int, mode: int, border: int,
                              stream=None) -> Plan:
    h = ctypes.c_void_p()
    _check(_native.load().resize_plan_create_border(ctypes.byref(h), in_h, in_w, out_h, out_w, mode, border,
                                                    _stream(stream)), "resize_plan_create_border")
    return Plan(h.value, in_h, in_w, out_h, out_w, mode, border)


def resize_plan_destroy(plan: Plan) -> None:
    plan.destroy()


def resize_plan_status(plan: Plan) -> int:
    st = ctypes.c_int(-1)
    _check(_native.load().resize_plan_status(plan.handle, ctypes.byref(st)), "resize_plan_status")
    return st.value


def resize_plan_set_tile(plan: Plan, kind: int, tile_rows: int, tile_cols: int) -> None:
    _check(_native.load().resize_plan_set_tile(plan.handle, kind, tile_rows, tile_cols), "resize_plan_set_tile")


def resize_plan_set_option(plan: Plan, option: int, value: int) -> None:
    _check(_native.load().resize_plan_set_option(plan.handle, option, value), "resize_plan_set_option")


def _hwc(t, name):
    """(H, W, C, pitch_bytes) of an HWC/HW tensor whose pixels are packed."""
    if t.dim() == 2:
        H, W = t.shape
        C = 1
        if t.stride(1) != 1:
            raise ValueError(f"{name}: columns must be contiguous")
    elif t.dim() == 3:
        H, W, C = t.shape
        if (C > 1 and t.stride(2) != 1) or t.stride(1) != C:
            raise ValueError(f"{name}: pixels must be packed (stride(1) == C, stride(2) == 1)")
    else:
        raise ValueError(f"{name}: expected HxW or HxWxC, got shape {tuple(t.shape)}")
    return H, W, C, t.stride(0) * t.element_size()


def resize_u8(plan: Plan, src, dst, mode: int | None = None, stream=None) -> None:
    """dst[:] = resize(src) for uint8 tensors (H, W[, C]) -> (OH, OW[, C])."""
    H, W, C, sp = _hwc(src, "src")
    OH, OW, C2, dp = _hwc(dst, "dst")
    if C2 != C:
        raise ValueError("src and dst channel counts differ")
    _check(_native.load().resize_u8(plan.handle, src.data_ptr(), sp, dst.data_ptr(), dp, H, W, C, OH, OW,
                                    plan.mode if mode is None else mode, _stream(stream)), "resize_u8")


def resize_u8_noalloc(src, dst, mode: int = RZ_LINEAR, stream=None) -> None:
    """dst[:] = resize(src) for uint8 tensors without a plan and without any
    device allocation (tables in the library's static device array; see
    include/gbresize.h for the size limit and the sharing rules)."""
    H, W, C, sp = _hwc(src, "src")
    OH, OW, C2, dp = _hwc(dst, "dst")
    if C2 != C:
        raise ValueError("src and dst channel counts differ")
    _check(_native.load().resize_u8_noalloc(src.data_ptr(), sp, dst.data_ptr(), dp, H, W, C, OH, OW, mode,
                                            _stream(stream)), "resize_u8_noalloc")


def resize_f32(plan: Plan, src, dst, mode: int | None = None, stream=None) -> None:
    """dst[:] = resize(src) for float32 tensors (H, W[, C]) -> (OH, OW[, C])."""
    H, W, C, sp = _hwc(src, "src")
    OH, OW, C2, dp = _hwc(dst, "dst")
    if C2 != C:
        raise ValueError("src and dst channel counts differ")
    _check(_native.load().resize_f32(plan.handle, src.data_ptr(), sp, dst.data_ptr(), dp, H, W, C, OH, OW,
                                     plan.mode if mode is None else mode, _stream(stream)), "resize_f32")


def _nhwc(t, name):
    """(N, H, W, C, pitch_bytes, batch_stride_bytes) of an NHWC tensor whose pixels are packed."""
    if t.dim() != 4:
        raise ValueError(f"{name}: expected NxHxWxC, got shape {tuple(t.shape)}")
    N, H, W, C = t.shape
    if (C > 1 and t.stride(3) != 1) or t.stride(2) != C:
        raise ValueError(f"{name}: pixels must be packed (stride(2) == C, stride(3) == 1)")
    es = t.element_size()
    return N, H, W, C, t.stride(1) * es, t.stride(0) * es


def _batch(fn_name, plan, src, dst, mode, stream):
    N, H, W, C, sp, sb = _nhwc(src, "src")
    N2, OH, OW, C2, dp, db = _nhwc(dst, "dst")
    if N2 != N or C2 != C:
        raise ValueError("src and dst batch or channel counts differ")
    _check(getattr(_native.load(), fn_name)(plan.handle, src.data_ptr(), sp, sb, dst.data_ptr(), dp, db, N, H, W, C,
                                            OH, OW, plan.mode if mode is None else mode, _stream(stream)), fn_name)


def resize_u8_batch(plan: Plan, src, dst, mode: int | None = None, stream=None) -> None:
    """dst[n] = resize(src[n]) for uint8 tensors (N, H, W, C) -> (N, OH, OW, C), one launch."""
    _batch("resize_u8_batch", plan, src, dst, mode, stream)


def resize_f32_batch(plan: Plan, src, dst, mode: int | None = None, stream=None) -> None:
    """dst[n] = resize(src[n]) for float32 tensors (N, H, W, C) -> (N, OH, OW, C), one launch."""
    _batch("resize_f32_batch", plan, src, dst, mode, stream)


def resize_wait_selftest(dev_status, limit_us: int, stream=None) -> None:
    """Launch the bounded-wait self-test: dev_status (a one-element int32 CUDA
    tensor) receives RZ_ERR_TIMEOUT when the wait gives up after limit_us."""
    _check(_native.load().resize_wait_selftest(dev_status.data_ptr(), limit_us, _stream(stream)),
           "resize_wait_selftest")


def make_epilogue(kind: int, batch: int = 1, src_batch_stride: int = 0, dst_batch_stride: int = 0,
                  mean=(0.0, 0.0, 0.0, 0.0), std=(1.0, 1.0, 1.0, 1.0), w3x3=None, wk=None) -> RzEpilogue:
    """An rz_epilogue; wk is a K x K weight array (odd K <= 7) for RZ_EPI_FILTER."""
    e = RzEpilogue()
    e.kind, e.batch = kind, batch
    e.src_batch_stride, e.dst_batch_stride = src_batch_stride, dst_batch_stride
    for i in range(4):
        e.mean[i] = float(mean[i]) if i < len(mean) else 0.0
        e.std[i] = float(std[i]) if i < len(std) else 1.0
    if w3x3 is not None:
        for i in range(9):
            e.w3x3[i] = float(w3x3[i])
    if wk is not None:
        rows = [list(r) for r in wk]
        e.ksize = len(rows)
        flat = [float(v) for r in rows for v in r]
        if len(flat) != e.ksize * e.ksize or e.ksize > 7:
            raise ValueError("wk must be a square array of at most 7 x 7 weights")
        for i, v in enumerate(flat):
            e.wk[i] = v
    return e


def resize_fused(plan: Plan, src, dst, epilogue: RzEpilogue, stream=None) -> None:
    """Resize with a fused epilogue.

    RZ_EPI_NORMALIZE_NCHW: src uint8 (N, H, W, C) or (H, W, C); dst float32
    (N, C, OH, OW) or (C, OH, OW).  RZ_EPI_FILTER3X3: src and dst float32
    (N, H, W, C) / (H, W, C) / (H, W).  RZ_EPI_GRAY_RGB / RZ_EPI_GRAY_BGR:
    src uint8 (N, H, W, C) or (H, W, C) with C = 3 or 4, dst uint8 (N, OH, OW)
    or (OH, OW), in the plan's mode.  The epilogue's batch and batch strides
    are filled in from the tensors.
    """
    import torch
    e = RzEpilogue.from_buffer_copy(epilogue)
    batched = src.dim() == 4
    s = src if batched else src.unsqueeze(0)
    mode = RZ_LINEAR
    if e.kind in (RZ_EPI_GRAY_RGB, RZ_EPI_GRAY_BGR):
        d = dst if dst.dim() == 3 else dst.unsqueeze(0)
        N, OH, OW = d.shape
        C = s.shape[3]
        if d.stride(2) != 1:
            raise ValueError("dst rows must be contiguous")
        dp = d.stride(1)
        dtype_code = RZ_U8
        mode = plan.mode
        if s.dtype != torch.uint8 or d.dtype != torch.uint8:
            raise ValueError("gray epilogue takes uint8 src and dst")
    elif e.kind == RZ_EPI_NORMALIZE_NCHW:
        d = dst if dst.dim() == 4 else dst.unsqueeze(0)
        N, C, OH, OW = d.shape
        if d.stride(3) != 1 or d.stride(1) != OH * d.stride(2):
            raise ValueError("dst planes must be rows of contiguous floats with planes stacked by rows")
        dp = d.stride(2) * 4
        dtype_code = RZ_U8
        if s.dtype != torch.uint8 or d.dtype != torch.float32:
            raise ValueError("normalise epilogue takes uint8 src and float32 dst")
    elif e.kind in (RZ_EPI_FILTER3X3, RZ_EPI_FILTER):
        if not batched and src.dim() == 2:
            s = src.unsqueeze(0).unsqueeze(-1)
            d = dst.unsqueeze(0).unsqueeze(-1)
        else:
            d = dst if dst.dim() == 4 else dst.unsqueeze(0)
        N, OH, OW, C = d.shape
        dp = d.stride(1) * 4
        dtype_code = RZ_F32
        if s.dtype != torch.float32 or d.dtype != torch.float32:
            raise ValueError("filter epilogues take float32 src and dst")
    else:
        raise ValueError(f"unknown epilogue kind {e.kind}")
    Nb, H, W, Cs = s.shape
    if Nb != N or Cs != C:
        raise ValueError("src and dst batch or channel counts differ")
    if (C > 1 and s.stride(3) != 1) or s.stride(2) != C:
        raise ValueError("src pixels must be packed")
    e.batch = N
    e.src_batch_stride = s.stride(0) * s.element_size()
    e.dst_batch_stride = d.stride(0) * d.element_size()
    _check(_native.load().resize_fused(plan.handle, s.data_ptr(), dtype_code, s.stride(1) * s.element_size(),
                                       d.data_ptr(), dp, H, W, C, OH, OW, mode, ctypes.byref(e),
                                       _stream(stream)), "resize_fused")


def filter2d_valid_f32(src, weights, dst, stream=None, kernel: int = RZ_FILTER_AUTO, status=None) -> None:
    """dst[:] = the K x K correlation of src over its valid region.

    src: float32 CUDA tensor (H, W) with contiguous rows; weights: float32
    CUDA tensor (K, K); dst: float32 CUDA tensor (H - K + 1, W - K + 1).
    kernel: RZ_FILTER_AUTO, RZ_FILTER_FP32 or RZ_FILTER_TENSOR; status:
    optional int32 CUDA tensor for the tensor-core kernel's time-outs.
    """
    if src.dim() != 2 or dst.dim() != 2 or src.stride(1) != 1 or dst.stride(1) != 1:
        raise ValueError("src and dst must be 2-D with contiguous rows")
    K = weights.shape[0]
    if weights.dim() != 2 or weights.shape[1] != K or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous K x K tensor")
    H, W = src.shape
    _check(_native.load().filter2d_valid_f32_ex(src.data_ptr(), src.stride(0) * 4, H, W, weights.data_ptr(), K,
                                                dst.data_ptr(), dst.stride(0) * 4, kernel,
                                                status.data_ptr() if status is not None else None, _stream(stream)),
           "filter2d_valid_f32")


def resize_copy_baseline(src, dst, flags: int = RZ_COPY_PDL | RZ_COPY_L2_PREFETCH, stream=None) -> None:
    """dst[:] = src, bytes moved by the library's 1:1 copy baseline kernel.

    src, dst: contiguous CUDA tensors of the same byte size (a multiple of
    16), 16-byte aligned, not overlapping.
    """
    if not (src.is_contiguous() and dst.is_contiguous()):
        raise ValueError("src and dst must be contiguous")
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes:
        raise ValueError("src and dst differ in byte size")
    _check(_native.load().resize_copy_baseline(src.data_ptr(), dst.data_ptr(), nbytes, flags, _stream(stream)),
           "resize_copy_baseline")


def make_jobs(srcs, dsts, device=None):
    """A device array of rz_job descriptors for resize_u8_multi from lists of
    uint8 HWC (or HW) CUDA tensors; returns (jobs tensor, C)."""
    import torch
    if len(srcs) != len(dsts):
        raise ValueError("srcs and dsts differ in length")
    arr = (_native.RzJob * max(1, len(srcs)))()
    C = None
    for k, (s, d) in enumerate(zip(srcs, dsts)):
        H, W, cs, sp = _hwc(s, "src")
        OH, OW, cd, dp = _hwc(d, "dst")
        if cs != cd or (C is not None and cs != C):
            raise ValueError("every job must have the same channel count")
        C = cs
        arr[k] = _native.RzJob(s.data_ptr(), d.data_ptr(), sp, dp, H, W, OH, OW)
    raw = bytes(memoryview(arr))[:ctypes.sizeof(_native.RzJob) * len(srcs)]
    dev = device if device is not None else (srcs[0].device if srcs else "cuda")
    jobs = torch.frombuffer(bytearray(raw), dtype=torch.uint8).to(dev) if raw else torch.empty(
        0, dtype=torch.uint8, device=dev)
    return jobs, (C or 1)


def resize_u8_multi(jobs, njobs: int, C: int, mode: int = RZ_LINEAR, status=None, stream=None) -> None:
    """Launch the jobs of a device job array (make_jobs) in one kernel;
    status: optional one-element int32 CUDA tensor receiving RZ_ERR_ARG when
    a job is invalid."""
    _check(_native.load().resize_u8_multi(jobs.data_ptr() if njobs else None, njobs, C, mode,
                                          status.data_ptr() if status is not None else None, _stream(stream)),
           "resize_u8_multi")


_torch = None
_MAP_DTYPES: dict = {}


def _with_torch():
    global _torch
    if _torch is None:
        import torch
        _MAP_DTYPES.update({torch.float32: RZ_F32, torch.bfloat16: RZ_BF16, torch.float16: RZ_F16})
        _torch = torch
    return _torch


def _map_dtype(t, name: str) -> int:
    code = _MAP_DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: expected float32, bfloat16 or float16, got {t.dtype}")
    return code


#: ctypes cuts what it stores in an int to 32 bits without an error.
_INT_MAX = 0x7FFFFFFF


def _int(v, name: str):
    if not -_INT_MAX <= v <= _INT_MAX:
        raise ValueError(f"{name}: {v} does not fit 32 bits")
    return v


def _map_of(t, name: str, shape=None):
    """((N, H, W, C), rz_map) of an (N, H, W, C) or (H, W, C) tensor whose pixels are packed; `shape`: what it must be."""
    dims = t.dim()
    if dims == 4:
        N, H, W, C = got = tuple(t.shape)
    elif dims == 3:
        H, W, C = t.shape
        N, got = 1, (1, H, W, C)
    else:
        raise ValueError(f"{name}: expected NxHxWxC or HxWxC, got shape {tuple(t.shape)}")
    if shape is not None and got != shape:
        raise ValueError(f"{name}: shape {got}, expected {shape}")
    if max(got) > _INT_MAX:
        raise ValueError(f"{name}: shape {got} past 2^31 - 1")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    es = t.element_size()
    if t.is_contiguous():
        return got, RzMap(t.data_ptr(), W * C * es, H * W * C * es)
    sn, sh, sw, sc = t.stride() if dims == 4 else (0, *t.stride())
    if t.numel() and ((C > 1 and sc != 1) or (W > 1 and sw != C)):
        raise ValueError(f"{name}: pixels must be packed (channels last)")
    return got, RzMap(t.data_ptr(), sh * es if H > 1 else W * C * es, sn * es if N > 1 else 0)


def _on_current_device(t, *others) -> None:
    """Kernels go to the current device, so every tensor of a call has to be there (as a plan's calls have to be on
    the plan's)."""
    device = t.get_device()
    for o in others:
        if o is not None and o.get_device() != device:
            raise ValueError("the tensors of a call are on different devices")
    if device != _torch._C._cuda_getDevice():
        raise ValueError(f"the tensors are on device {device}, which is not the current one")


def _floats(t, name: str, shape):
    """Pointer of a packed float32 CUDA tensor of that shape (None: a null pointer)."""
    if t is None:
        return None
    if t.dtype is not _torch.float32 or t.shape != shape or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous float32 CUDA tensor of shape {shape}")
    return t.data_ptr()


def _drop_of(p, seed, offset=0) -> RzDrop:
    return RzDrop(p, seed & 0xFFFFFFFFFFFFFFFF, offset & 0xFFFFFFFFFFFFFFFF)


def _stream_at(stream, t) -> int:
    """The call's stream: `stream`, or the current one of the tensor's device
    (its handle alone: a stream object costs as much as a launch)."""
    return _torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else _stream(stream)


def _with_workspace(call, workspace, query, d, like, stream) -> int:
    """call(pointer, bytes, stream) with the given workspace, or with query(d)
    bytes from torch's allocator that belong to the call's stream and go back
    once it is queued (without a tensor around them, which costs as much as
    two launches)."""
    s = _stream_at(stream, like)
    if workspace is not None:
        if not (workspace.is_cuda and workspace.get_device() == like.get_device() and workspace.is_contiguous()):
            raise ValueError("workspace: expected a contiguous CUDA tensor on the device of the others")
        return call(workspace.data_ptr(), workspace.numel() * workspace.element_size(), s)
    nbytes = query(d)
    if nbytes == 0:
        return call(None, 0, s)
    c = _torch._C
    p = c._cuda_cudaCachingAllocator_raw_alloc(nbytes, s)
    try:
        return call(p, nbytes, s)
    finally:
        c._cuda_cudaCachingAllocator_raw_delete(p)


def map_dropout(x, y, p: float, seed: int, offset: int = 0, residual=None, stream=None) -> None:
    """y[:] = dropout(x) + residual with the counter-based mask of (p, seed,
    offset); called on dy without a residual it is the gradient towards x.
    Any shape, packed or in the (N, H, W, C) layout of the other maps; y may
    be x or the residual."""
    _with_torch()
    dtype = _map_dtype(x, "x")
    both = (x, y) if residual is None else (x, y, residual)
    for t in both[1:]:
        if t.dtype is not x.dtype or t.shape != x.shape or not t.is_cuda:
            raise ValueError("x, y and residual differ in dtype or shape, or are not CUDA tensors")
    if not x.is_cuda:
        raise ValueError("x: expected a CUDA tensor")
    _on_current_device(x, y, residual)
    drop = _drop_of(p, seed, offset)
    if all(t.is_contiguous() for t in both):
        # any shape whose elements follow one another, their number past 32 bits among them
        r = None if residual is None else residual.data_ptr()
        rc = _native.load().map_dropout_packed(x.data_ptr(), r, y.data_ptr(), x.numel(), dtype, drop, _stream_at(stream, x))
    else:
        shape = _map_of(x, "x")[0]
        maps = [_map_of(t, name)[1] for t, name in zip(both, ("x", "y", "residual"))]
        rc = _native.load().map_dropout(maps[0], maps[2] if residual is not None else None, maps[1], *shape, dtype, drop,
                                        _stream_at(stream, x))
    _check(rc, "map_dropout")


def _norm_workspace(d) -> int:
    n = ctypes.c_size_t(0)
    _check(_native.load().map_group_norm_workspace(d, ctypes.byref(n)), "map_group_norm_workspace")
    return n.value


def map_group_norm_workspace(x, groups: int) -> int:
    """Bytes of workspace that map_group_norm and map_group_norm_grad need on a map like x."""
    _with_torch()
    return _norm_workspace(RzNorm(*_map_of(x, "x")[0], _int(groups, "groups"), _map_dtype(x, "x"), RZ_ACT_NONE, 1.0))


def map_group_norm(x, y, groups: int, gamma=None, beta=None, mean=None, rstd=None, act: int = RZ_ACT_NONE,
                   eps: float = 1e-5, drop=None, workspace=None, stream=None) -> None:
    """y[:] = dropout(act(group_norm(x))) on (N, H, W, C) or (H, W, C) maps.

    gamma, beta: float32 (C,) or None; mean, rstd: float32 (N, groups) written
    for the gradient, or None; act: RZ_ACT_*; drop: (p, seed, offset) or None;
    workspace: a CUDA tensor of map_group_norm_workspace(x, groups) bytes, or
    None to take one from torch's allocator."""
    _with_torch()
    shape, mx = _map_of(x, "x")
    _on_current_device(x, y, gamma, beta, mean, rstd)
    my = _map_of(y, "y", shape)[1]
    if y.dtype is not x.dtype:
        raise ValueError("x and y differ in dtype")
    d = RzNorm(*shape, _int(groups, "groups"), _map_dtype(x, "x"), _int(act, "act"), eps)
    channels, stats = (shape[3],), (shape[0], groups)
    dr = None if drop is None else _drop_of(*drop)
    g, b = _floats(gamma, "gamma", channels), _floats(beta, "beta", channels)
    m, r = _floats(mean, "mean", stats), _floats(rstd, "rstd", stats)
    f = _native.load().map_group_norm
    _check(_with_workspace(lambda w, n, st: f(d, dr, mx, my, g, b, m, r, w, n, st), workspace, _norm_workspace, d, x,
                           stream), "map_group_norm")


def map_group_norm_grad(dy, x, dx, groups: int, gamma=None, beta=None, mean=None, rstd=None, dgamma=None, dbeta=None,
                        act: int = RZ_ACT_NONE, eps: float = 1e-5, drop=None, workspace=None, stream=None) -> None:
    """dx[:], dgamma[:] and dbeta[:] (either may be None) from dy, with the
    arguments of the map_group_norm call and the mean and rstd it wrote."""
    _with_torch()
    shape, mx = _map_of(x, "x")
    _on_current_device(x, dy, dx, gamma, beta, mean, rstd, dgamma, dbeta)
    md, mo = _map_of(dy, "dy", shape)[1], _map_of(dx, "dx", shape)[1]
    if dy.dtype is not x.dtype or dx.dtype is not x.dtype:
        raise ValueError("x, dy and dx differ in dtype")
    d = RzNorm(*shape, _int(groups, "groups"), _map_dtype(x, "x"), _int(act, "act"), eps)
    channels, stats = (shape[3],), (shape[0], groups)
    dr = None if drop is None else _drop_of(*drop)
    g, b = _floats(gamma, "gamma", channels), _floats(beta, "beta", channels)
    m, r = _floats(mean, "mean", stats), _floats(rstd, "rstd", stats)
    dg, db = _floats(dgamma, "dgamma", channels), _floats(dbeta, "dbeta", channels)
    f = _native.load().map_group_norm_grad
    _check(_with_workspace(lambda w, n, st: f(d, dr, md, mx, mo, g, b, m, r, dg, db, w, n, st), workspace,
                           _norm_workspace, d, x, stream), "map_group_norm_grad")


def _resample_of(src, dst, names):
    _with_torch()
    (Ns, H, W, C), ms = _map_of(src, names[0])
    (N, OH, OW, C2), md = _map_of(dst, names[1])
    if C2 != C or Ns not in (1, N):
        raise ValueError(f"{names[0]} and {names[1]} differ in channels or images")
    return RzResample(N, Ns, H, W, OH, OW, C, _map_dtype(dst, names[1]), _map_dtype(src, names[0])), ms, md


def resize_map(src, dst, base=None, stream=None) -> None:
    """dst[:] = base + the bilinear resize of src, on (N, H, W, C) or (H, W, C)
    maps with any number of channels.  A src of one image serves every image of
    dst (a position table); it may be float32 where dst is 16-bit."""
    d, ms, md = _resample_of(src, dst, ("src", "dst"))
    _on_current_device(dst, src, base)
    mb = None
    if base is not None:
        if base.dtype is not dst.dtype:
            raise ValueError("base and dst differ in dtype")
        mb = _map_of(base, "base", (d.N, d.out_h, d.out_w, d.C))[1]
    _check(_native.load().resize_map(d, ms, mb, md, _stream_at(stream, dst)), "resize_map")


def _resample_workspace(d) -> int:
    n = ctypes.c_size_t(0)
    _check(_native.load().resize_map_grad_workspace(d, ctypes.byref(n)), "resize_map_grad_workspace")
    return n.value


def resize_map_grad_workspace(ddst, dsrc) -> int:
    """Bytes of workspace that resize_map_grad needs for these maps."""
    return _resample_workspace(_resample_of(dsrc, ddst, ("dsrc", "ddst"))[0])


def resize_map_grad(ddst, dsrc, workspace=None, stream=None) -> None:
    """dsrc[:] = the gradient of resize_map towards src, from ddst; summed over
    the images where dsrc has one."""
    d, ms, md = _resample_of(dsrc, ddst, ("dsrc", "ddst"))
    _on_current_device(ddst, dsrc)
    f = _native.load().resize_map_grad
    _check(_with_workspace(lambda w, n, st: f(d, md, ms, w, n, st), workspace, _resample_workspace, d, ddst, stream),
           "resize_map_grad")


class Texture:
    """Owns an ``rz_tex`` handle (a texture object over a uint8 image); the
    image tensor is kept alive with it."""

    def __init__(self, src):
        H, W, C, pitch = _hwc(src, "src")
        h = ctypes.c_void_p()
        _check(_native.load().resize_texture_create(ctypes.byref(h), src.data_ptr(), pitch, H, W, C),
               "resize_texture_create")
        self.handle, self.src, self.C = h.value, src, C

    def resize(self, dst, stream=None) -> None:
        """dst[:] = the hardware-filtered bilinear resize of the image."""
        OH, OW, C, pitch = _hwc(dst, "dst")
        if C != self.C:
            raise ValueError("dst channels differ from the image's")
        _check(_native.load().resize_texture_u8(self.handle, dst.data_ptr(), pitch, OH, OW, _stream(stream)),
               "resize_texture_u8")

    def destroy(self) -> None:
        if self.handle:
            h, self.handle = self.handle, None
            _check(_native.load().resize_texture_destroy(h), "resize_texture_destroy")

    def __del__(self):
        try:
            if self.handle:
                _native.load().resize_texture_destroy(self.handle)
                self.handle = None
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.destroy()


def resize_texture_create(src) -> Texture:
    return Texture(src)


def resize_u8_host(plan: Plan, host_src, host_dst, dev_src, dev_dst, stream=None) -> None:
    """Host -> device copy, resize, device -> host copy, queued on one stream.

    host_src/host_dst are CPU tensors (page-locked for asynchronous copies);
    dev_src/dev_dst are the caller's device buffers of the same shapes.
    """
    H, W, C, hsp = _hwc(host_src, "host_src")
    OH, OW, _, hdp = _hwc(host_dst, "host_dst")
    _, _, _, dsp = _hwc(dev_src, "dev_src")
    _, _, _, ddp = _hwc(dev_dst, "dev_dst")
    _check(_native.load().resize_u8_host(plan.handle, host_src.data_ptr(), hsp, host_dst.data_ptr(), hdp,
                                         dev_src.data_ptr(), dsp, dev_dst.data_ptr(), ddp, H, W, C, OH, OW,
                                         plan.mode, _stream(stream)), "resize_u8_host")


def resize_axis_table(n_in: int, n_out: int, mode: int = RZ_LINEAR):
    """Host-only sampling table of one axis: (ofs int32, w_q11 int32, u float32) numpy arrays."""
    import numpy as np
    ofs = np.zeros(n_out, np.int32)
    w = np.zeros(n_out, np.int32)
    u = np.zeros(n_out, np.float32)
    _check(_native.load().resize_axis_table(n_in, n_out, mode, ofs.ctypes.data, w.ctypes.data, u.ctypes.data),
           "resize_axis_table")
    return ofs, w, u


def resize_axis_table_border(n_in: int, n_out: int, mode: int, border: int):
    """resize_axis_table under a border rule."""
    import numpy as np
    ofs = np.zeros(n_out, np.int32)
    w = np.zeros(n_out, np.int32)
    u = np.zeros(n_out, np.float32)
    _check(_native.load().resize_axis_table_border(n_in, n_out, mode, border, ofs.ctypes.data, w.ctypes.data,
                                                   u.ctypes.data), "resize_axis_table_border")
    return ofs, w, u


def resize_strerror(code: int) -> str:
    return _native.load().resize_strerror(code).decode()


def resize_last_cuda_error() -> int:
    return _native.load().resize_last_cuda_error()
