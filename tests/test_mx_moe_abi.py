"""Refusals and sizes of the MXFP4 type and the mixture-of-experts entry points
on the CPU (fake device addresses: only where no GPU is visible, as nothing
may be enqueued), and the references' own pins."""
import ctypes

import numpy as np
import pytest

import mx_ref as R
from quantized_matmul_ggml_amd import binding as B

no_gpu = pytest.mark.skipif(__import__("torch").cuda.device_count() > 0,
                            reason="fake device addresses: host-only validation checks run where no GPU is visible")

BASE = 0x7F0000000000
W, X, Y, U, D, IDS, WTS, WS = (BASE + (i << 32) for i in range(8))


def _ref(*ds):
    return [ctypes.byref(d) if d is not None else None for d in ds]


def _mx(K=2048, M=64, addr=W, pitch=None):
    return B.make_desc(B.MXFP4, K, M, B.row_size(B.MXFP4, K) if pitch is None else pitch, addr)


def _f32(ne0, ne1, addr):
    return B.make_desc(B.F32, ne0, ne1, 4 * ne0, addr)


def _bf16(K, N, addr=X):
    return B.make_desc(B.BF16, K, N, 2 * K, addr)


def test_row_size(qmm_lib):
    for K in (0, 32, 64, 96, 512, 544, 2048, 5632):
        assert qmm_lib.row_size(B.MXFP4, K) == R.row_size("mxfp4", K)
    assert qmm_lib.row_size(B.MXFP4, 512) == 17 * 16       # no padding
    assert qmm_lib.row_size(B.MXFP4, 48) == 0 and qmm_lib.row_size(B.MXFP4, -32) == 0
    assert qmm_lib.record_size(B.MXFP4) == 0


def test_reference_quantizer_by_hand():
    """One block worked out by hand: amax 7 gives e = 0; ties go to the even
    code, 7 saturates at 6, signs are kept."""
    w = np.zeros((1, 32), np.float32)
    w[0, :10] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, -1.6]
    rows = R.quantize_mxfp4(w)
    codes = [7, 0, 2, 2, 4, 4, 6, 6, 8, 8 + 3]
    assert rows[0, 0] == 127 and list(rows[0, 16:26]) == codes
    assert np.array_equal(R.values(rows, "mxfp4", 32)[0, :10], [6, 0, 1, 1, 2, 2, 4, 4, -0.0, -1.5])
    w[0, 31] = 2.0 ** -3
    w[0, 0] = 2.0 ** 10
    rows = R.quantize_mxfp4(w)
    assert rows[0, 0] == 127 + 8 and rows[0, 16] == 6
    assert R.quantize_mxfp4(np.zeros((1, 32), np.float32))[0, 0] == 0


@no_gpu
def test_gemv_and_quantize_reject(qmm_lib):
    call = B.call_raw
    assert call("qmm_gemv", _mx(K=2040), _f32(2040, 1, X), _f32(64, 1, Y)) == B.ERR_SHAPE
    assert call("qmm_gemv", _mx(), _f32(2048, 9, X), _f32(64, 9, Y)) == B.ERR_SHAPE
    assert call("qmm_gemv", _mx(addr=W + 8), _f32(2048, 1, X), _f32(64, 1, Y)) == B.ERR_LAYOUT
    assert call("qmm_gemv", _mx(pitch=1072), _f32(2048, 1, X), _f32(64, 1, Y)) == B.ERR_LAYOUT
    assert call("qmm_gemv", _mx(pitch=(1 << 26) + 16), _f32(2048, 1, X), _f32(64, 1, Y + (1 << 34))) == B.ERR_UNSUPPORTED
    # packed activations of a GEMV stay Q8_0, with integer weights
    assert call("qmm_gemv", _mx(), _mx(M=1, addr=X), _f32(64, 1, Y)) == B.ERR_TYPE
    assert call("qmm_gemv", _mx(), B.make_desc(B.Q8_0, 2048, 1, 2176, X), _f32(64, 1, Y)) == B.ERR_TYPE
    assert call("qmm_gemv_swiglu", _mx(), _mx(addr=U), B.make_desc(B.Q8_0, 2048, 1, 2176, X), _f32(64, 1, Y)) == B.ERR_TYPE
    assert call("qmm_gemv_swiglu", _mx(), B.make_desc(B.Q4_0, 2048, 64, 1152, U), _f32(2048, 1, X), _f32(64, 1, Y)) == B.ERR_TYPE
    assert B.call_batch_raw([(_mx(), B.make_desc(B.Q8_0, 2048, 1, 2176, X), _f32(64, 1, Y))]) == B.ERR_TYPE
    # bf16 sources are for MXFP4 only, 16-byte aligned
    q4 = B.make_desc(B.Q4_0, 2048, 4, 1152, W)
    assert call("qmm_quantize", _bf16(2048, 4), q4) == B.ERR_TYPE
    assert call("qmm_quantize", _bf16(2048, 4, X + 8), _mx(M=4)) == B.ERR_LAYOUT
    assert call("qmm_quantize", B.make_desc(B.F16, 2048, 4, 4096, X), _mx(M=4)) == B.ERR_TYPE
    assert call("qmm_quantize", _f32(2048, 4, W + 1024), _mx(M=4)) == B.ERR_ALIAS
    rule = qmm_lib.lib().qmm_quantize_rule
    assert rule(*_ref(_f32(2048, 4, X), _mx(M=4)), 1, None) == B.ERR_TYPE      # amax / 7 is a Q4 rule
    for f, a in (("qmm_records_to_rows", (ctypes.c_void_p(X), ctypes.byref(_mx()))),
                 ("qmm_rows_to_records", (ctypes.byref(_mx()), ctypes.c_void_p(X)))):
        assert getattr(qmm_lib.lib(), f)(*a, None) == B.ERR_TYPE
    assert call("qmm_gemv", _mx(M=0, addr=0), _f32(2048, 1, X), _f32(0, 1, 0)) == B.OK


@no_gpu
def test_gemm_reject(qmm_lib):
    call = B.call_raw
    x, y = _mx(M=512, addr=X), _f32(64, 512, Y)
    assert call("qmm_gemm", B.make_desc(B.Q4_0, 2048, 64, 1152, W), x, y) == B.ERR_TYPE
    assert call("qmm_gemm", B.make_desc(B.F16, 2048, 64, 4096, W), x, y) == B.ERR_TYPE
    assert call("qmm_gemm", _mx(), B.make_desc(B.Q8_0, 2048, 512, 2176, X), y) == B.ERR_TYPE
    assert call("qmm_gemm", _mx(), _mx(K=1024, M=512, addr=X), y) == B.ERR_SHAPE
    assert call("qmm_gemm", _mx(), _mx(M=512, addr=X + 8), y) == B.ERR_LAYOUT
    assert call("qmm_gemm", _mx(), x, _f32(64, 512, X)) == B.ERR_ALIAS
    assert call("qmm_gemm", _mx(pitch=1 << 24), x, _f32(64, 512, Y)) == B.ERR_UNSUPPORTED
    assert call("qmm_gemm_swiglu", _mx(), _mx(addr=U), x, y) == B.ERR_TYPE
    item = B.QmmGemmItem(*(ctypes.pointer(d) for d in (_mx(), x, y)))
    assert qmm_lib.lib().qmm_gemm_batch((B.QmmGemmItem * 1)(item), 1, None) == B.ERR_TYPE
    assert qmm_lib.lib().qmm_gemm_workspace_size(*_ref(_mx(), x)) == 0
    assert qmm_lib.lib().qmm_gemm_noalloc(*_ref(_mx(), x, y), B.NOALLOC_SCRATCH_BYTES + 16, None) == B.ERR_SCRATCH
    assert call("qmm_gemm", _mx(), _mx(M=0, addr=0), _f32(64, 0, 0)) == B.OK


def _ex(K, M, E, addr, type_=B.MXFP4, pitch2=None):
    t = B.make_desc(type_, K, M, B.row_size(type_, K), addr, n_dims=3)
    t.ne[2] = E
    t.nb[2] = B.row_size(type_, K) * M if pitch2 is None else pitch2
    return t


@no_gpu
def test_moe_rejects(qmm_lib):
    f = qmm_lib.lib().qmm_moe_swiglu
    K, F, M, E, N, k = 256, 128, 64, 8, 4, 2

    def call(gate=None, up=None, down=None, x=None, y=None, ids=IDS, wts=WTS, k=k, ws=WS, size=1 << 20, N=N):
        a = [gate or _ex(K, F, E, W), up or _ex(K, F, E, U), down or _ex(F, M, E, D), x or _f32(K, N, X)]
        return f(*_ref(*a), ctypes.c_void_p(ids), ctypes.c_void_p(wts), k, *_ref(y or _f32(M, N, Y)), ctypes.c_void_p(ws),
                 size, None)

    g = _ex(K, F, E, W)
    assert f(None, *_ref(g, g, _f32(K, N, X)), None, None, k, None, None, 0, None) == B.ERR_NULL
    need = qmm_lib.lib().qmm_moe_workspace_size(*_ref(g, _f32(K, N, X)), k)
    assert need == N * k * 4 * 192                      # one group of four blocks per pair
    assert qmm_lib.lib().qmm_moe_workspace_size(*_ref(g, _f32(K, 9, X)), k) == 0
    assert qmm_lib.lib().qmm_moe_workspace_size(None, None, k) == 0
    two = B.make_desc(B.MXFP4, K, F, B.row_size(B.MXFP4, K), W)
    assert call(gate=two) == B.ERR_UNSUPPORTED          # not three dimensions
    assert call(gate=_ex(K, F, E, W, B.Q4_0)) == B.ERR_TYPE                    # mixed types
    f16 = B.make_desc(B.F16, K, F, 2 * K, W, n_dims=3)
    f16.ne[2] = E
    assert call(gate=f16) == B.ERR_TYPE
    assert call(up=_ex(K, F, E + 1, U)) == B.ERR_SHAPE
    assert call(up=_ex(K, F + 1, E, U)) == B.ERR_SHAPE
    assert call(down=_ex(F + 32, M, E, D)) == B.ERR_SHAPE
    assert call(gate=_ex(K, F, 0, W)) == B.ERR_SHAPE
    assert call(x=_f32(K + 32, N, X)) == B.ERR_SHAPE
    assert call(x=_f32(K, 9, X), y=_f32(M, 9, Y)) == B.ERR_SHAPE
    assert call(k=0) == B.ERR_SHAPE and call(k=17) == B.ERR_SHAPE
    assert call(y=_f32(M + 1, N, Y)) == B.ERR_SHAPE
    assert call(x=B.make_desc(B.BF16, K, N, 2 * K, X)) == B.ERR_TYPE
    assert call(y=B.make_desc(B.F16, M, N, 2 * M, Y)) == B.ERR_TYPE
    assert call(gate=_ex(K, F, E, W, pitch2=B.row_size(B.MXFP4, K) * F - 16)) == B.ERR_LAYOUT
    assert call(gate=_ex(K, F, E, W, pitch2=B.row_size(B.MXFP4, K) * F + 8)) == B.ERR_LAYOUT
    assert call(gate=_ex(K, F, E, W + 4)) == B.ERR_LAYOUT
    assert call(ids=0) == B.ERR_NULL and call(wts=0) == B.ERR_NULL and call(ws=0) == B.ERR_NULL
    assert call(ids=IDS + 2) == B.ERR_LAYOUT and call(wts=WTS + 1) == B.ERR_LAYOUT and call(ws=WS + 8) == B.ERR_LAYOUT
    assert call(size=need - 1) == B.ERR_SCRATCH
    for at in (W + 4096, U, D + 64, X, IDS, WTS + 28, WS):
        assert call(y=_f32(M, N, at)) == B.ERR_ALIAS
    for at in (W, D, X, IDS - 16, WTS):
        assert call(ws=at) == B.ERR_ALIAS
    assert call(gate=_ex(K, F, E, W, pitch2=1 << 62)) == B.ERR_UNSUPPORTED
    assert call(x=_f32(K, 0, 0), y=_f32(M, 0, 0), N=0) == B.OK


@no_gpu
def test_route_rejects(qmm_lib):
    f = qmm_lib.lib().qmm_moe_route

    def call(l, k=2, rule=1, ids=IDS, wts=WTS):
        return f(*_ref(l), k, rule, ctypes.c_void_p(ids), ctypes.c_void_p(wts), None)

    l = _f32(64, 8, X)
    assert call(None) == B.ERR_NULL
    assert call(l, rule=2) == B.ERR_UNSUPPORTED and call(l, rule=-1) == B.ERR_UNSUPPORTED
    assert call(l, k=0) == B.ERR_SHAPE and call(l, k=17) == B.ERR_SHAPE and call(_f32(4, 8, X), k=5) == B.ERR_SHAPE
    assert call(_f32(1025, 8, X)) == B.ERR_UNSUPPORTED
    assert call(_bf16(64, 8)) == B.ERR_TYPE
    assert call(l, ids=0) == B.ERR_NULL and call(l, wts=0) == B.ERR_NULL
    assert call(l, ids=IDS + 1) == B.ERR_LAYOUT and call(l, wts=WTS + 2) == B.ERR_LAYOUT
    assert call(l, ids=WTS + 32) == B.ERR_ALIAS and call(l, ids=X) == B.ERR_ALIAS and call(l, wts=X + 64) == B.ERR_ALIAS
    assert call(_f32(64, 0, 0), ids=0, wts=0) == B.OK
