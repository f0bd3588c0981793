"""ctypes binding of libqmm (include/qmm.h): argument marshalling only.

Every computation runs in the HIP kernels of libqmm.so; this module only
builds ``qmm_tensor`` descriptors from torch tensors (device memory and the
current stream come from torch) and turns non-zero status codes into
exceptions.  There is no CPU fallback: if the library is missing or a tensor
is not on the GPU, the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

# qmm_type
F32, F16, BF16, Q8_0, Q4_0, Q8_B64, Q4_B64, MXFP4 = 0, 1, 2, 3, 4, 5, 6, 7
TYPE_NAMES = {F32: "F32", F16: "F16", BF16: "BF16", Q8_0: "Q8_0", Q4_0: "Q4_0",
              Q8_B64: "Q8_B64", Q4_B64: "Q4_B64",
              MXFP4: "MXFP4"}

# qmm_status
OK, ERR_NULL, ERR_TYPE, ERR_SHAPE, ERR_LAYOUT, ERR_ALIAS, ERR_UNSUPPORTED, ERR_DEVICE, ERR_SCRATCH = \
    0, -1, -2, -3, -4, -5, -6, -7, -8
NOALLOC_SCRATCH_BYTES = 16 << 20

EXPORTS = ("qmm_row_size", "qmm_quantize", "qmm_quantize_rule", "qmm_dequantize", "qmm_gemv", "qmm_gemv_batch",
           "qmm_gemv_swiglu", "qmm_gemm", "qmm_gemm_ws", "qmm_gemm_noalloc", "qmm_gemm_workspace_size", "qmm_gemm_batch", "qmm_gemm_swiglu", "qmm_record_size", "qmm_records_to_rows",
           "qmm_rows_to_records", "qmm_moe_route", "qmm_moe_workspace_size", "qmm_moe_swiglu", "qmm_stream_read", "qmm_clock_probe", "qmm_wall_clock_khz", "qmm_strerror")
GEMV_BATCH_MAX = 8
MOE_MAX_TOKENS, MOE_MAX_TOP_K, MOE_MAX_ROUTED = 8, 16, 1024
# qmm_route_rule
ROUTE_ALL, ROUTE_CHOSEN = 0, 1


class QmmTensor(ctypes.Structure):
    """Mirror of ``qmm_tensor`` (ne/nb convention: ne[0] contiguous, nb in bytes)."""
    _fields_ = [("type", ctypes.c_int32), ("n_dims", ctypes.c_int32),
                ("ne", ctypes.c_int64 * 4), ("nb", ctypes.c_uint64 * 4),
                ("data", ctypes.c_void_p)]


_PACK = struct.Struct("=ii4q4QQ").pack      # the fields of QmmTensor
_ELEM = {F32: 4, F16: 2, BF16: 2}
_DTYPE = {F32: torch.float32, F16: torch.float16, BF16: torch.bfloat16}
_U64 = (1 << 64) - 1
assert struct.calcsize("=ii4q4QQ") == ctypes.sizeof(QmmTensor)


class QmmGemvItem(ctypes.Structure):
    """Mirror of ``qmm_gemv_item``."""
    _fields_ = [("w", ctypes.POINTER(QmmTensor)), ("x_f32", ctypes.POINTER(QmmTensor)),
                ("y_f32", ctypes.POINTER(QmmTensor))]


class QmmGemmItem(ctypes.Structure):
    """Mirror of ``qmm_gemm_item``."""
    _fields_ = [("w", ctypes.POINTER(QmmTensor)), ("x_bf16", ctypes.POINTER(QmmTensor)),
                ("y_f32", ctypes.POINTER(QmmTensor))]


class QmmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {strerror(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """Load libqmm.so from the package directory (build it with build.py)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m quantized_matmul_ggml_amd.build` "
                "(hipcc, gfx950); there is no fallback implementation")
        h = ctypes.CDLL(LIB_PATH)
        # descriptors: packed bytes (_PACK), or ctypes.byref of a QmmTensor
        P = ctypes.c_void_p
        h.qmm_row_size.argtypes = [ctypes.c_int32, ctypes.c_int64]
        h.qmm_row_size.restype = ctypes.c_size_t
        h.qmm_quantize.argtypes = [P, P, ctypes.c_void_p]
        h.qmm_quantize_rule.argtypes = [P, P, ctypes.c_int32, ctypes.c_void_p]
        h.qmm_quantize_rule.restype = ctypes.c_int
        h.qmm_dequantize.argtypes = [P, P, ctypes.c_void_p]
        h.qmm_gemv.argtypes = [P, P, P, ctypes.c_void_p]
        h.qmm_gemm.argtypes = [P, P, P, ctypes.c_void_p]
        h.qmm_gemm_ws.argtypes = [P, P, P, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
        h.qmm_gemm_ws.restype = ctypes.c_int
        h.qmm_gemm_noalloc.argtypes = [P, P, P, ctypes.c_size_t, ctypes.c_void_p]
        h.qmm_gemm_noalloc.restype = ctypes.c_int
        h.qmm_gemm_workspace_size.argtypes = [P, P]
        h.qmm_gemm_workspace_size.restype = ctypes.c_size_t
        h.qmm_gemm_batch.argtypes = [ctypes.POINTER(QmmGemmItem), ctypes.c_int32, ctypes.c_void_p]
        h.qmm_gemm_batch.restype = ctypes.c_int
        h.qmm_gemm_swiglu.argtypes = [P, P, P, P, ctypes.c_void_p]
        h.qmm_gemm_swiglu.restype = ctypes.c_int
        h.qmm_gemv_swiglu.argtypes = [P, P, P, P, ctypes.c_void_p]
        h.qmm_gemv_swiglu.restype = ctypes.c_int
        h.qmm_record_size.argtypes = [ctypes.c_int32]
        h.qmm_record_size.restype = ctypes.c_size_t
        h.qmm_records_to_rows.argtypes = [ctypes.c_void_p, P, ctypes.c_void_p]
        h.qmm_records_to_rows.restype = ctypes.c_int
        h.qmm_rows_to_records.argtypes = [P, ctypes.c_void_p, ctypes.c_void_p]
        h.qmm_rows_to_records.restype = ctypes.c_int
        h.qmm_gemv_batch.argtypes = [ctypes.POINTER(QmmGemvItem), ctypes.c_int32, ctypes.c_void_p]
        h.qmm_gemv_batch.restype = ctypes.c_int
        V, I = ctypes.c_void_p, ctypes.c_int32
        h.qmm_moe_route.argtypes = [P, I, I, V, V, V]
        h.qmm_moe_route.restype = ctypes.c_int
        h.qmm_moe_workspace_size.argtypes = [P, P, I]
        h.qmm_moe_workspace_size.restype = ctypes.c_size_t
        h.qmm_moe_swiglu.argtypes = [P, P, P, P, V, V, I, P, V, ctypes.c_size_t, V]
        h.qmm_moe_swiglu.restype = ctypes.c_int
        for f in ("qmm_quantize", "qmm_dequantize", "qmm_gemv", "qmm_gemm"):
            getattr(h, f).restype = ctypes.c_int
        h.qmm_stream_read.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_void_p]
        h.qmm_stream_read.restype = ctypes.c_int
        h.qmm_clock_probe.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                      ctypes.c_void_p]
        h.qmm_clock_probe.restype = ctypes.c_int
        h.qmm_wall_clock_khz.argtypes = []
        h.qmm_wall_clock_khz.restype = ctypes.c_int64
        h.qmm_strerror.argtypes = [ctypes.c_int]
        h.qmm_strerror.restype = ctypes.c_char_p
        _lib = h
    return _lib


def strerror(status: int) -> str:
    return lib().qmm_strerror(status).decode()


def row_size(type_: int, K: int) -> int:
    return int(lib().qmm_row_size(type_, K))


_row_bytes = functools.lru_cache(row_size)      # 0.5 us less, for the checks of every call


def make_desc(type_: int, ne0: int, ne1: int, nb1: int, data_ptr: int, n_dims: int = 2,
              nb0: int | None = None) -> QmmTensor:
    """A raw descriptor (used directly by the boundary tests)."""
    if nb0 is None:
        nb0 = _ELEM.get(type_, 0)
    nb2 = nb1 * (ne1 if ne1 > 1 else 1) & _U64
    # one packed copy: filling the fields one by one costs several microseconds
    return QmmTensor.from_buffer_copy(_PACK(type_, n_dims, ne0, ne1, 1, 1, nb0 & _U64, nb1 & _U64, nb2, nb2, data_ptr or 0))


# The library checks a descriptor's sizes against each other, not against the
# memory behind them: neither a single row's pitch nor the end of the last row.
_DATA = "data must hold M rows of K packed weights, each contiguous"


@dataclass
class Weight:
    """A weight matrix W (ne = [K, M]): M rows of K weights on the GPU.

    data is uint8 (M, pitch) for quantized rows (Q8_0, Q4_0, Q8_B64, Q4_B64, MXFP4) in the row-planar layout of
    include/qmm.h, or float16 (M, >= K) for F16 rows."""
    data: torch.Tensor
    type: int
    K: int
    M: int

    @property
    def pitch(self) -> int:
        return self.data.stride(0) * self.data.element_size()

    def desc(self) -> QmmTensor:
        return QmmTensor.from_buffer_copy(self._desc())

    def _desc(self) -> bytes:
        d, M = self.data, self.M
        (pitch, step), (rows, cols), es = d.stride(), d.shape, d.element_size()
        if M and (step != 1 or rows < M or (M == 1 or cols != pitch) and cols * es < _row_bytes(self.type, self.K)):
            raise ValueError(_DATA)
        pitch *= es
        nb2 = pitch * M if M > 1 else pitch
        return _PACK(self.type, 2, self.K, M, 1, 1, _ELEM.get(self.type, 0), pitch, nb2, nb2, d.data_ptr())

    def rows(self, r0: int, r1: int) -> "Weight":
        """Row-range view [r0, r1): no copy, same pitch."""
        return Weight(self.data[r0:r1], self.type, self.K, r1 - r0)


def _need_gpu(*ts: torch.Tensor) -> int:
    """The one GPU the tensors are on."""
    dev = ts[0].get_device()
    for t in ts:
        d = t.get_device()
        if d < 0:
            raise ValueError("libqmm operates on GPU tensors only")
        if d != dev:
            raise ValueError("the tensors of a call must be on one GPU")
    return dev


def _need_bytes(t: torch.Tensor, nbytes: int, what: str):
    """Refuses a buffer that is not one run of at least nbytes bytes (a strided
    or expanded tensor's memory is not all its own, nor as much as its elements)."""
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{what} holds fewer than {nbytes} bytes")


def _row_pitch(pitch: int, row_bytes: int) -> int:
    """The pitch of packed rows to make: a single row's, too, holds the row (the
    library does not look at it)."""
    if pitch < row_bytes:
        raise ValueError(f"a pitch of {pitch} bytes is below the row's {row_bytes}")
    return pitch


def _dense_desc(t: torch.Tensor, type_: int) -> QmmTensor:
    """2-D row-major torch tensor (rows, cols) -> ne = [cols, rows]."""
    return QmmTensor.from_buffer_copy(_dense(t, type_))


def _dense(t: torch.Tensor, type_: int) -> bytes:
    """_dense_desc's bytes.  The element type is checked here: a descriptor
    says nothing of how many bytes its memory holds, so that the library would
    read or write past the end of a narrower tensor."""
    if t.dtype is not _DTYPE[type_]:
        raise ValueError(f"expected a {_DTYPE[type_]} tensor, not {t.dtype}")
    shape, es = t.shape, _ELEM[type_]
    if len(shape) != 2:
        raise ValueError("expected a 2-D tensor")
    rows, cols = shape
    if rows == 0 or cols == 0:          # empty: strides are meaningless
        pitch = cols * es
    else:
        pitch, step = t.stride()
        if step != 1:
            raise ValueError("rows must be contiguous (stride 1 along the last dimension)")
        pitch *= es
    nb2 = pitch * rows if rows > 1 else pitch
    return _PACK(type_, 2, cols, rows, 1, 1, es, pitch, nb2, nb2, t.data_ptr())


# The current stream's handle without building a Stream object (2.8 us less per
# call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
# The current device, for callers that hold a tensor of a GPU (so that torch's
# own check that the GPU is initialised is not needed).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    return _raw_stream(torch.cuda.current_device()) if stream is None else stream.cuda_stream


def _on(stream):
    """Makes `stream` the current one (None: leaves it), for what a call does
    through torch before its launch: a copy made on any other stream would run
    in no order with the launch, and its memory could be handed out again
    before the launch has read it."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


# Memory that a call makes for itself belongs to the stream it runs on: what the
# allocator hands out for another stream may still be in use there by earlier
# work, in no order with this call's.
def _output(stream, device, dtype, *shape) -> torch.Tensor:
    """A tensor to return.  The caller goes on with it on the current stream,
    and may let go of it while that still reads."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(*shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(device))
    return out


def _workspace(stream, device, nbytes: int) -> torch.Tensor:
    """Scratch memory that is let go of when the call returns: work that takes
    it over on its stream runs after the call's."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _launch(dev: int, stream, name: str, *args):
    """Calls entry point `name` on GPU dev, on `stream` or that GPU's current
    stream; raises what it refuses."""
    if stream is None:
        handle = _raw_stream(dev)
    elif stream.device_index == dev:
        handle = stream.cuda_stream
    else:
        raise ValueError(f"a stream of GPU {stream.device_index} cannot run work on tensors of GPU {dev}")
    fn = getattr(_lib or lib(), name)
    if dev == _current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != OK:
        raise QmmError(status, name)


def _check(status: int, where: str):
    if status != OK:
        raise QmmError(status, where)


QUANT_DEFAULT, QUANT_Q4_AMAX7 = 0, 1


def quantize(w: torch.Tensor, type_: int, *, pitch: int | None = None, rule: int = QUANT_DEFAULT,
             stream=None) -> Weight:
    """Quantize fp32 rows w (M, K) on the GPU into Q8_0 / Q4_0 rows, or their
    64-weight-block variants Q8_B64 / Q4_B64 (rule: QUANT_DEFAULT, or
    QUANT_Q4_AMAX7 for the symmetric amax/7 Q4 rule), or MXFP4 rows (fp32 or
    bf16 w)."""
    dev = _need_gpu(w)
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("quantize takes float32 rows (or bfloat16 ones, for MXFP4)")
    M, K = w.shape
    rs = _row_bytes(type_, K)
    pitch = rs if pitch is None else _row_pitch(pitch, rs)
    out = _output(stream, w.device, torch.uint8, M, pitch)
    if pitch > rs:
        with _on(stream):
            out[:, rs:].zero_()
    wt = Weight(out, type_, K, M)
    _launch(dev, stream, "qmm_quantize_rule", _dense(w, BF16 if w.dtype == torch.bfloat16 else F32), wt._desc(), rule)
    return wt


def dequantize(w: Weight, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W' as fp32 (M, K)."""
    if out is None:
        out = _output(stream, w.data.device, torch.float32, w.M, w.K)
    _launch(_need_gpu(w.data, out), stream, "qmm_dequantize", w._desc(), _dense(out, F32))
    return out


def f16_weight(w16: torch.Tensor) -> Weight:
    """Wrap float16 rows (M, K) as an F16 weight."""
    _need_gpu(w16)
    assert w16.dtype == torch.float16
    return Weight(w16, F16, w16.shape[1], w16.shape[0])


def gemv(w: Weight, x, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y (N, M) fp32 = x (N, K) times W'^T; 1 <= N <= 8.  x is fp32 (N, K), or
    a Q8_0 Weight of N rows (activations quantized with quantize()) for the
    integer-activation path."""
    xt, n, xd = (x.data, x.M, x._desc()) if isinstance(x, Weight) else (x, x.shape[0], _dense(x, F32))
    if out is None:
        out = _output(stream, xt.device, torch.float32, n, w.M)
    _launch(_need_gpu(w.data, xt, out), stream, "qmm_gemv", w._desc(), xd, _dense(out, F32))
    return out


def gemv_batch(items, *, stream=None) -> list:
    """Several GEMVs in one launch: items = [(Weight, x, out or None), ...]
    sharing the weight type, K and N; x is fp32 (N, K) in every item, or a
    Q8_0 Weight of N rows in every item (the integer-activation path).
    Returns the outputs."""
    descs, keep, outs, tensors = [], [], [], []
    for w, x, out in items:
        xt, n, xd = (x.data, x.M, x.desc()) if isinstance(x, Weight) else (x, x.shape[0], _dense_desc(x, F32))
        if out is None:
            out = _output(stream, xt.device, torch.float32, n, w.M)
        tensors += [w.data, xt, out]
        wd, yd = w.desc(), _dense_desc(out, F32)
        keep += [wd, xd, yd]
        descs.append(QmmGemvItem(ctypes.pointer(wd), ctypes.pointer(xd), ctypes.pointer(yd)))
        outs.append(out)
    arr = (QmmGemvItem * max(1, len(descs)))(*descs)
    if tensors:
        _launch(_need_gpu(*tensors), stream, "qmm_gemv_batch", arr, len(descs))
    else:
        _check(lib().qmm_gemv_batch(arr, 0, _stream(stream)), "qmm_gemv_batch")
    return outs


def gemv_swiglu(w_gate: Weight, w_up: Weight, x, *, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """h (N, M) fp32 = Swish(x W_gate'^T) * (x W_up'^T), one fused launch; 1 <= N <= 8.
    x is fp32 (N, K), or a Q8_0 Weight of N rows for the integer-activation path."""
    xt, n, xd = (x.data, x.M, x._desc()) if isinstance(x, Weight) else (x, x.shape[0], _dense(x, F32))
    if out is None:
        out = _output(stream, xt.device, torch.float32, n, w_gate.M)
    _launch(_need_gpu(w_gate.data, w_up.data, xt, out), stream, "qmm_gemv_swiglu", w_gate._desc(), w_up._desc(), xd,
            _dense(out, F32))
    return out


def record_size(type_: int) -> int:
    """Bytes of one GGUF-style block record (18 for Q4_0, 34 for Q8_0, else 0)."""
    return int(lib().qmm_record_size(type_))


def records_to_rows(records: torch.Tensor, type_: int, K: int, M: int, *, pitch: int | None = None,
                    stream=None) -> Weight:
    """Packed rows (a Weight) from M * K/32 block records (uint8 device tensor)."""
    dev = _need_gpu(records)
    rs = _row_bytes(type_, K)
    pitch = rs if pitch is None else _row_pitch(pitch, rs)
    _need_bytes(records, M * (K // 32) * record_size(type_), "records")
    out = _output(stream, records.device, torch.uint8, M, pitch)
    with _on(stream):
        out.zero_()
    wt = Weight(out, type_, K, M)
    _launch(dev, stream, "qmm_records_to_rows", records.data_ptr(), wt._desc())
    return wt


def rows_to_records(w: Weight, *, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The M * K/32 block records of a quantized Weight (uint8 device tensor)."""
    n = w.M * (w.K // 32) * record_size(w.type)
    if out is None:
        out = _output(stream, w.data.device, torch.uint8, n)
    _need_bytes(out, n, "out")
    _launch(_need_gpu(w.data, out), stream, "qmm_rows_to_records", w._desc(), out.data_ptr())
    return out


def gemm_workspace_size(w: Weight, x) -> int:
    """Bytes of workspace qmm_gemm_ws uses to split K for these shapes (0: no
    split, as for every packed x)."""
    return int(lib().qmm_gemm_workspace_size(w._desc(), x._desc() if isinstance(x, Weight) else _dense(x, BF16)))


def gemm(w: Weight, x, *, out: torch.Tensor | None = None, workspace="auto",
         stream=None) -> torch.Tensor:
    """y (N, M) fp32 = x (N, K) bf16 times W'^T on the bf16 matrix cores, or, for
    an MXFP4 w, an MXFP4 Weight x of N rows on the scaled matrix instructions.

    workspace: "auto" allocates the split-K workspace the shapes call for (a
    torch allocation, so it is graph-capture safe), None runs without one
    (qmm_gemm), or a uint8 device tensor to use as is."""
    xt, n, xd = (x.data, x.M, x._desc()) if isinstance(x, Weight) else (x, x.shape[0], _dense(x, BF16))
    if out is None:
        out = _output(stream, xt.device, torch.float32, n, w.M)
    dev, wd, yd = _need_gpu(w.data, xt, out), w._desc(), _dense(out, F32)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        n = int(lib().qmm_gemm_workspace_size(wd, xd))
        workspace = _workspace(stream, xt.device, n) if n else None
    elif workspace is not None:
        _need_bytes(workspace, 0, "workspace")
    if workspace is None:
        _launch(dev, stream, "qmm_gemm", wd, xd, yd)
    else:
        _need_gpu(out, workspace)
        _launch(dev, stream, "qmm_gemm_ws", wd, xd, yd, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def gemm_noalloc(w: Weight, x, out: torch.Tensor, *, workspace_bytes: int | None = None,
                 stream=None) -> torch.Tensor:
    """qmm_gemm_noalloc: the GEMM with its split-K partial sums in the
    library's static scratch array (no allocation in the call; `out` is the
    caller's).  workspace_bytes defaults to the full split of these shapes.  x
    is bf16 or packed, as in gemm."""
    xt, xd = (x.data, x._desc()) if isinstance(x, Weight) else (x, _dense(x, BF16))
    dev, wd = _need_gpu(w.data, xt, out), w._desc()
    if workspace_bytes is None:
        workspace_bytes = int(lib().qmm_gemm_workspace_size(wd, xd))
    _launch(dev, stream, "qmm_gemm_noalloc", wd, xd, _dense(out, F32), workspace_bytes)
    return out


def gemm_swiglu(w_gate: Weight, w_up: Weight, x: torch.Tensor, *, out: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """h (N, M) fp32 = Swish(x W_gate'^T) * (x W_up'^T) for bf16 x (N, K), one fused launch."""
    if out is None:
        out = _output(stream, x.device, torch.float32, x.shape[0], w_gate.M)
    _launch(_need_gpu(w_gate.data, w_up.data, x, out), stream, "qmm_gemm_swiglu", w_gate._desc(), w_up._desc(),
            _dense(x, BF16), _dense(out, F32))
    return out


def gemm_batch(items, *, stream=None) -> list:
    """Several prefill GEMMs in one launch: items = [(Weight, x (N, K) bf16, out or None), ...]
    sharing the weight type, K and N.  Returns the outputs."""
    descs, keep, outs, tensors = [], [], [], []
    for w, x, out in items:
        if out is None:
            out = _output(stream, x.device, torch.float32, x.shape[0], w.M)
        tensors += [w.data, x, out]
        wd, xd, yd = w.desc(), _dense_desc(x, BF16), _dense_desc(out, F32)
        keep += [wd, xd, yd]
        descs.append(QmmGemmItem(ctypes.pointer(wd), ctypes.pointer(xd), ctypes.pointer(yd)))
        outs.append(out)
    arr = (QmmGemmItem * max(1, len(descs)))(*descs)
    if tensors:
        _launch(_need_gpu(*tensors), stream, "qmm_gemm_batch", arr, len(descs))
    else:
        _check(lib().qmm_gemm_batch(arr, 0, _stream(stream)), "qmm_gemm_batch")
    return outs


@dataclass
class Experts:
    """E weight matrices of one type and shape (ne = [K, M, E]): data is uint8
    (E, M, pitch), quantized rows of K weights as in Weight."""
    data: torch.Tensor
    type: int
    K: int
    M: int

    def desc(self) -> QmmTensor:
        return QmmTensor.from_buffer_copy(self._desc())

    def _desc(self) -> bytes:
        d, M = self.data, self.M
        (apart, pitch, step), (E, rows, cols), es = d.stride(), d.shape, d.element_size()
        if M and (step != 1 or rows < M or (M == 1 or cols != pitch) and cols * es < _row_bytes(self.type, self.K)):
            raise ValueError(_DATA)
        nb2 = apart * es
        return _PACK(self.type, 3, self.K, M, E, 1, 0, pitch * es, nb2, nb2 * E, d.data_ptr())

    def expert(self, e: int) -> Weight:
        """Expert e's matrix: no copy."""
        return Weight(self.data[e], self.type, self.K, self.M)


def quantize_experts(w: torch.Tensor, type_: int, *, stream=None) -> Experts:
    """Quantize fp32 matrices w (E, M, K) on the GPU into Experts (MXFP4: or bf16
    ones).  Matrices whose rows are not evenly spaced are copied first."""
    if w.dim() != 3:
        raise ValueError("expected a 3-D tensor")
    E, M, K = w.shape
    with _on(stream):
        rows = w.reshape(E * M, K)
    q = quantize(rows, type_, stream=stream)
    return Experts(q.data.view(E, M, q.data.shape[1]), type_, K, M)


def moe_route(logits: torch.Tensor, top_k: int, *, rule: int = ROUTE_CHOSEN, stream=None) -> tuple:
    """(ids int32, weights fp32), each (N, top_k): every token's top_k experts of
    its logits (N, E) fp32, largest first, with softmax weights over all
    experts (ROUTE_ALL) or over the chosen ones (ROUTE_CHOSEN).  Experts
    masked by -inf are never chosen; empty slots hold id -1 and weight 0."""
    if logits.dtype != torch.float32 or logits.dim() != 2:
        raise ValueError("logits must be float32 (N, E)")
    dev, n = _need_gpu(logits), logits.shape[0]
    ids = _output(stream, logits.device, torch.int32, n, top_k)
    weights = _output(stream, logits.device, torch.float32, n, top_k)
    _launch(dev, stream, "qmm_moe_route", _dense(logits, F32), top_k, rule, ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_workspace_size(w_gate: Experts, x: torch.Tensor, top_k: int) -> int:
    """Bytes of workspace qmm_moe_swiglu needs for these shapes."""
    return int(lib().qmm_moe_workspace_size(w_gate._desc(), _dense(x, F32), top_k))


def moe_swiglu(w_gate: Experts, w_up: Experts, w_down: Experts, x: torch.Tensor, ids: torch.Tensor,
               weights: torch.Tensor, *, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y (N, M) fp32: the sum over each token's slots of weights times the
    SwiGLU block of expert ids (int32), both (N, top_k) and contiguous;
    x (N, K) fp32, N <= 8.  workspace: a uint8 device tensor of at least
    moe_workspace_size bytes, or None to allocate one (graph-capture safe)."""
    if ids.dtype != torch.int32 or weights.dtype != torch.float32 or x.dtype != torch.float32:
        raise ValueError("ids must be int32, weights and x float32")
    if ids.dim() != 2 or x.dim() != 2 or ids.shape != weights.shape or ids.shape[0] != x.shape[0] or not (ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError("ids and weights must be contiguous and (N, top_k)")
    top_k = ids.shape[1]
    if out is None:
        out = _output(stream, x.device, torch.float32, x.shape[0], w_down.M)
    elif out.dtype != torch.float32:
        raise ValueError("out must be float32")
    gd, xd = w_gate._desc(), _dense(x, F32)
    if workspace is None:
        workspace = _workspace(stream, x.device, int(lib().qmm_moe_workspace_size(gd, xd, top_k)))
    else:
        _need_bytes(workspace, 0, "workspace")
    dev = _need_gpu(w_gate.data, w_up.data, w_down.data, x, ids, weights, out, workspace)
    _launch(dev, stream, "qmm_moe_swiglu", gd, w_up._desc(), w_down._desc(), xd, ids.data_ptr(), weights.data_ptr(), top_k,
            _dense(out, F32), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def call_batch_raw(triples, count=None, stream: int = 0) -> int:
    """qmm_gemv_batch with hand-made descriptors [(w, x, y), ...]; returns the status."""
    items = [QmmGemvItem(*(ctypes.pointer(d) if d is not None else None for d in t)) for t in triples]
    arr = (QmmGemvItem * max(1, len(items)))(*items)
    n = len(items) if count is None else count
    return lib().qmm_gemv_batch(arr, n, ctypes.c_void_p(stream))


def call_raw(name: str, *descs: QmmTensor, stream: int = 0) -> int:
    """Call an entry point with hand-made descriptors; returns the status."""
    fn = getattr(lib(), name)
    return fn(*[ctypes.byref(d) if d is not None else None for d in descs], ctypes.c_void_p(stream))


def stream_read(src: torch.Tensor, sink: torch.Tensor, *, nbytes: int | None = None, workgroups: int = 1024,
                stream=None) -> None:
    """qmm_stream_read over the first nbytes (default: all) of the device
    tensor src; sink: an int32 device tensor of at least `workgroups` words."""
    dev = _need_gpu(src, sink)
    n = src.numel() * src.element_size() if nbytes is None else nbytes
    _need_bytes(src, n, "src")
    _need_bytes(sink, 4 * workgroups, "sink")
    _launch(dev, stream, "qmm_stream_read", src.data_ptr(), n, sink.data_ptr(), workgroups)


def clock_probe(workgroups: int = 256, iters: int = 20000, mode: int = 0) -> float:
    """Shader clock in MHz under a dependent chain on every wave (mode 0:
    binary32 FMAs, mode 1: bf16 matrix instructions), from the device's
    shader-clock and constant-rate counters; synchronizes."""
    out = torch.zeros(8 * workgroups, dtype=torch.int64, device="cuda")
    _check(lib().qmm_clock_probe(ctypes.c_void_p(out.data_ptr()), workgroups, iters, mode, _stream(None)),
           "qmm_clock_probe")
    d = out.view(-1, 2).cpu()
    wall_khz = int(lib().qmm_wall_clock_khz())
    if wall_khz <= 0:
        raise QmmError(wall_khz, "qmm_wall_clock_khz")
    return float(d[:, 0].sum()) / float(d[:, 1].sum()) * wall_khz / 1e3


def mfma_probe(mode: int, workgroups: int = 256, iters: int = 4000) -> dict:
    """The block-GEMM inner-loop probe (qmm_clock_probe modes 2-4) on every
    CU: multiply-add rate in TFLOP/s over the waves' own clocks, and shader
    clock cycles per round (four 32 x 32 x 32 tile-blocks) per wave: the mean
    over waves and the slowest wave (waves sharing a SIMD do not run in
    lockstep, so the SIMD's rate is that of its last wave to finish)."""
    out = torch.zeros(8 * workgroups, dtype=torch.int64, device="cuda")
    _check(lib().qmm_clock_probe(ctypes.c_void_p(out.data_ptr()), workgroups, iters, mode, _stream(None)),
           "qmm_clock_probe")
    d = out.view(-1, 2).cpu().double()
    wall_khz = int(lib().qmm_wall_clock_khz())
    if wall_khz <= 0:
        raise QmmError(wall_khz, "qmm_wall_clock_khz")
    seconds = float(d[:, 1].mean()) / (wall_khz * 1e3)
    flops = 4.0 * workgroups * iters * 4 * 2 * 32 * 32 * 32
    return {"tflops": flops / seconds / 1e12, "cycles_per_round": float(d[:, 0].mean()) / iters,
            "cycles_per_round_max": float(d[:, 0].max()) / iters}
