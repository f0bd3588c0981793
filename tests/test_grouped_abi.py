"""Refusals and sizes of the grouped products, the layer of many tokens and the
low-rank adapters on the CPU (fake device addresses: only where no GPU is
visible, as nothing may be enqueued)."""
import ctypes

import pytest

from quantized_matmul_ggml_amd import binding as B

no_gpu = pytest.mark.skipif(__import__("torch").cuda.device_count() > 0,
                            reason="fake device addresses: host-only validation checks run where no GPU is visible")

BASE = 0x7F0000000000
W, X, Y, U, D, IDS, WTS, WS, OFF, ORD, PLACE = (BASE + (i << 32) for i in range(11))
TOP = (1 << 64) - 4


def _ref(*ds):
    return [ctypes.byref(d) if d is not None else None for d in ds]


def _v(p):
    return ctypes.c_void_p(p)


def _dense(type_, cols, rows, at, pitch=None):
    return B.make_desc(type_, cols, rows, (4 if type_ == B.F32 else 2) * cols if pitch is None else pitch, at)


def _ex(K, M, E, at, type_=B.Q4_0, pitch=None, pitch2=None, n_dims=3):
    p = B.row_size(type_, K) if pitch is None else pitch
    t = B.make_desc(type_, K, M, p, at, n_dims=n_dims)
    t.ne[2], t.nb[2] = E, p * max(M, 1) if pitch2 is None else pitch2
    return t


def _adapters(cols, rows, L, at, pitch=None, apart=None, type_=B.BF16):
    t = B.make_desc(type_, cols, rows, 2 * cols if pitch is None else pitch, at, n_dims=3)
    t.ne[2], t.nb[2] = L, (2 * cols if pitch is None else pitch) * max(rows, 1) if apart is None else apart
    return t


# ------------------------------------------------------------------ grouping

def test_group_workspace(qmm_lib):
    size = B.moe_group_workspace_size
    assert [size(n, 8) for n in (-1, 0, 1, 65536)] == [0, 0, 0, 0]
    assert size(65537, 8) == size(1 << 30, 8) == 64 * 9 * 4
    assert size(65537, 0) == 0 and size(65537, 1025) == 0 and size(1 << 31, 8) == 0 and size(65537, 1024) == 64 * 1025 * 4


@no_gpu
def test_group_rejects(qmm_lib):
    f = qmm_lib.lib().qmm_moe_group

    def call(ids=IDS, n=100, E=8, off=OFF, order=ORD, place=PLACE, ws=0, size=0):
        return f(_v(ids), n, E, _v(off), _v(order), _v(place), _v(ws), size, None)

    assert call(n=-1) == B.ERR_SHAPE and call(E=0) == B.ERR_SHAPE and call(E=-3) == B.ERR_SHAPE
    assert call(n=1 << 31) == B.ERR_UNSUPPORTED and call(E=1025) == B.ERR_UNSUPPORTED
    for name in ("ids", "off", "order", "place"):
        assert call(**{name: 0}) == B.ERR_NULL, name
        assert call(**{name: IDS + (9 << 34) + 2}) == B.ERR_LAYOUT, name
        assert call(**{name: TOP}) == B.ERR_UNSUPPORTED, name
    big = dict(n=65537, ws=WS, size=64 * 9 * 4)
    assert call(**{**big, "ws": 0}) == B.ERR_NULL and call(**{**big, "ws": WS + 4}) == B.ERR_LAYOUT
    assert call(**{**big, "size": 64 * 9 * 4 - 1}) == B.ERR_SCRATCH
    ends = {"ids": 4 * 65537, "off": 36, "order": 4 * 65537, "place": 4 * 65537, "ws": 64 * 9 * 4}
    at = {"ids": IDS, "off": OFF, "order": ORD, "place": PLACE, "ws": WS}
    for a in ends:
        for b in ends:
            if a != b:
                assert call(**{**big, a: at[b]}) == B.ERR_ALIAS, (a, b)
                if a != "ws":
                    assert call(**{**big, a: at[b] + ends[b] - 4}) == B.ERR_ALIAS, (a, b)
    assert call(n=0, off=0) == B.ERR_NULL
    assert call() == B.ERR_DEVICE and call(n=0, ids=0, order=0, place=0) == B.ERR_DEVICE      # past the checks: no GPU here


# ------------------------------------------------------------------ products

@no_gpu
@pytest.mark.parametrize("pair", [False, True])
def test_grouped_rejects(qmm_lib, pair):
    K, M, E, N, R, k = 256, 96, 8, 20, 40, 2
    h = qmm_lib.lib()

    def call(w=None, up=None, x=None, y=None, off=OFF, order=ORD, k=k):
        w, x, y = w or _ex(K, M, E, W), x or _dense(B.BF16, K, N, X), y or _dense(B.F32, M, R, Y)
        if pair:
            return h.qmm_gemm_grouped_swiglu(*_ref(w, up or _ex(K, M, E, U), x), _v(off), _v(order), k, *_ref(y), None)
        return h.qmm_gemm_grouped(*_ref(w, x), _v(off), _v(order), k, *_ref(y), None)

    one, x, y = _ex(K, M, E, W), _dense(B.BF16, K, N, X), _dense(B.F32, M, R, Y)
    for null in range(4 if pair else 3):
        ds = [one, one, x, y] if pair else [one, x, y]
        ds[null] = None
        f = h.qmm_gemm_grouped_swiglu if pair else h.qmm_gemm_grouped
        assert f(*_ref(*ds[:-1]), _v(OFF), _v(ORD), k, *_ref(ds[-1]), None) == B.ERR_NULL, null
    assert call(w=_ex(K, M, E, W, n_dims=2)) == B.ERR_UNSUPPORTED
    f16 = B.make_desc(B.F16, K, M, 2 * K, W, n_dims=3)
    f16.ne[2], f16.nb[2] = E, 2 * K * M
    assert call(w=f16) == B.ERR_TYPE
    for t in (B.F32, B.F16, B.Q8_0):
        assert call(x=B.make_desc(t, K, N, B.row_size(t, K), X)) == B.ERR_TYPE, t
    assert call(y=_dense(B.F16, M, R, Y)) == B.ERR_TYPE
    assert call(x=_dense(B.BF16, K + 32, N, X)) == B.ERR_SHAPE
    assert call(y=_dense(B.F32, M + 1, R, Y)) == B.ERR_SHAPE
    assert call(w=_ex(K, M, 0, W)) == B.ERR_SHAPE
    assert call(k=0) == B.ERR_SHAPE and call(k=-1) == B.ERR_SHAPE
    assert call(order=0) == B.ERR_SHAPE                     # 20 tokens, 40 rows
    assert call(x=_dense(B.BF16, K, N, X + 8)) == B.ERR_LAYOUT
    assert call(w=_ex(K, M, E, W + 4)) == B.ERR_LAYOUT
    assert call(w=_ex(K, M, E, W, pitch2=B.row_size(B.Q4_0, K) * M - 16)) == B.ERR_LAYOUT
    assert call(off=0) == B.ERR_NULL
    assert call(off=OFF + 2) == B.ERR_LAYOUT and call(order=ORD + 1) == B.ERR_LAYOUT
    assert call(off=TOP) == B.ERR_UNSUPPORTED and call(order=TOP) == B.ERR_UNSUPPORTED
    if pair:
        assert call(up=_ex(K, M, E, U, B.Q8_0)) == B.ERR_TYPE
        assert call(up=_ex(K, M + 32, E, U)) == B.ERR_SHAPE and call(up=_ex(K, M, E + 1, U)) == B.ERR_SHAPE
        assert call(y=_dense(B.F32, M, R, U + 64)) == B.ERR_ALIAS
    last = W + E * M * B.row_size(B.Q4_0, K) - 16
    for at in (W, last, X, X + 2 * K * N - 16, OFF, OFF + 4 * E, ORD, ORD + 4 * R - 4):
        assert call(y=_dense(B.F32, M, R, at)) == B.ERR_ALIAS, hex(at)
    # limits: experts, rows, pitches, the reach of picked and of ordered rows, the grid
    big = dict(order=0, y=_dense(B.F32, M, 1 << 31, Y), x=_dense(B.BF16, K, 1 << 31, X))
    assert call(w=_ex(K, M, 1025, W), up=_ex(K, M, 1025, U)) == B.ERR_UNSUPPORTED
    assert call(**big) == B.ERR_UNSUPPORTED
    assert call(w=_ex(K, M, E, W, pitch=1 << 24)) == B.ERR_UNSUPPORTED
    assert call(x=_dense(B.BF16, K, 128, X, pitch=1 << 24), y=_dense(B.F32, M, R, Y)) == B.ERR_UNSUPPORTED
    assert call(x=_dense(B.BF16, K, 40, X, pitch=1 << 24), order=0) == B.ERR_UNSUPPORTED
    wide = (1 << 28) + 32
    assert call(w=_ex(wide, 1, 1, W), up=_ex(wide, 1, 1, U), x=_dense(B.BF16, wide, 1, X), y=_dense(B.F32, 1, 1, Y), order=0) == B.ERR_UNSUPPORTED
    tall = dict(w=_ex(32, 1 << 28, 1, W), up=_ex(32, 1 << 28, 1, U))
    for n, status in ((64, B.ERR_DEVICE), (1024, B.ERR_UNSUPPORTED), (1 << 16, B.ERR_UNSUPPORTED)):       # 2^23 tiles of 128 x 128
        assert call(**tall, x=_dense(B.BF16, 32, n, X), y=_dense(B.F32, 1 << 28, n, Y + (1 << 48)), order=0) == status, n
    # nothing to do, and what is left to the GPU
    assert call(y=_dense(B.F32, M, 0, 0), off=0, order=0, x=_dense(B.BF16, K, 0, 0)) == B.OK
    assert call(w=_ex(K, 0, E, 0), up=_ex(K, 0, E, 0), y=_dense(B.F32, 0, R, 0), off=0) == B.OK
    assert call() == B.ERR_DEVICE and call(y=_dense(B.BF16, M, R, Y + 2)) == B.ERR_DEVICE
    assert call(x=_dense(B.BF16, K, R, X), order=0) == B.ERR_DEVICE
    assert call(x=_dense(B.BF16, K, 0, 0)) == B.ERR_DEVICE            # every picked row is zeros


# --------------------------------------------------------------------- layer

@no_gpu
def test_layer_rejects(qmm_lib):
    K, F, M, E, N, k = 256, 128, 66, 8, 50, 2
    h = qmm_lib.lib()

    def call(gate=None, up=None, down=None, x=None, y=None, ids=IDS, wts=WTS, k=k, ws=WS, size=1 << 24):
        a = [gate or _ex(K, F, E, W), up or _ex(K, F, E, U), down or _ex(F, M, E, D), x or _dense(B.BF16, K, N, X)]
        return h.qmm_moe_gemm_swiglu(*_ref(*a), _v(ids), _v(wts), k, *_ref(y or _dense(B.F32, M, N, Y)), _v(ws), size, None)

    g, d, x, y = _ex(K, F, E, W), _ex(F, M, E, D), _dense(B.BF16, K, N, X), _dense(B.F32, M, N, Y)
    size = lambda g, d, x, k: h.qmm_moe_gemm_workspace_size(*_ref(g, d, x), k)
    up256 = lambda n: (n + 255) // 256 * 256
    R = N * k
    need = up256(4 * (E + 1)) + 2 * up256(4 * R) + up256(2 * R * F) + up256(4 * R * 68)
    assert size(g, d, x, k) == need
    assert size(None, d, x, k) == size(g, None, x, k) == size(g, d, None, k) == size(g, d, x, 0) == size(g, d, x, 17) == 0
    assert size(g, d, _dense(B.BF16, K, 0, 0), k) == 0 and size(g, _ex(F, 0, E, 0), x, k) == 0
    for null in range(5):
        ds = [g, g, d, x, y]
        ds[null] = None
        assert h.qmm_moe_gemm_swiglu(*_ref(*ds[:4]), _v(IDS), _v(WTS), k, *_ref(ds[4]), _v(WS), 1 << 24, None) == B.ERR_NULL, null
    assert call(gate=_ex(K, F, E, W, B.Q8_0)) == B.ERR_TYPE and call(down=_ex(F, M, E, D, B.Q8_0)) == B.ERR_TYPE
    assert call(x=_dense(B.F32, K, N, X)) == B.ERR_TYPE and call(y=_dense(B.F16, M, N, Y)) == B.ERR_TYPE
    assert call(up=_ex(K, F + 32, E, U)) == B.ERR_SHAPE and call(down=_ex(F + 32, M, E, D)) == B.ERR_SHAPE
    assert call(down=_ex(F, M, E + 1, D)) == B.ERR_SHAPE and call(x=_dense(B.BF16, K + 32, N, X)) == B.ERR_SHAPE
    assert call(k=0) == B.ERR_SHAPE and call(k=17) == B.ERR_SHAPE
    assert call(y=_dense(B.F32, M + 1, N, Y)) == B.ERR_SHAPE and call(y=_dense(B.F32, M, N + 1, Y)) == B.ERR_SHAPE
    assert call(ids=0) == B.ERR_NULL and call(wts=0) == B.ERR_NULL and call(ws=0) == B.ERR_NULL
    assert call(ids=IDS + 2) == B.ERR_LAYOUT and call(wts=WTS + 1) == B.ERR_LAYOUT and call(ws=WS + 8) == B.ERR_LAYOUT
    assert call(size=need - 1) == B.ERR_SCRATCH and call(size=0) == B.ERR_SCRATCH
    assert call(ids=TOP) == B.ERR_UNSUPPORTED and call(wts=TOP) == B.ERR_UNSUPPORTED
    assert call(ws=(1 << 64) - 16, size=need) == B.ERR_UNSUPPORTED
    for at in (W, U + 64, D, X, IDS, WTS + 4 * R - 4, WS, WS + need - 4):
        assert call(y=_dense(B.F32, M, N, at)) == B.ERR_ALIAS, hex(at)
    for at in (W, U, D, X, IDS, WTS, IDS - 16):
        assert call(ws=at) == B.ERR_ALIAS, hex(at)
    # 2^31 rows of slots, h rows of 2^24 bytes, workspaces beyond the address space
    assert call(x=_dense(B.BF16, 32, 1 << 28, X), gate=_ex(32, F, E, W), up=_ex(32, F, E, U), k=8,
                y=_dense(B.F32, M, 1 << 28, Y)) == B.ERR_UNSUPPORTED
    F2 = 1 << 23
    assert call(gate=_ex(32, F2, 1, W), up=_ex(32, F2, 1, U), down=_ex(F2, 8, 1, D), x=_dense(B.BF16, 32, 1, X), k=1,
                y=_dense(B.F32, 8, 1, Y)) == B.ERR_UNSUPPORTED
    assert call(x=_dense(B.BF16, K, 0, 0), y=_dense(B.F32, M, 0, 0), ids=0, wts=0, ws=0, size=0) == B.OK
    assert call(down=_ex(F, 0, E, 0), y=_dense(B.F32, 0, N, 0), ids=0, wts=0, ws=0, size=0) == B.OK
    assert call(size=need) == B.ERR_DEVICE


# ------------------------------------------------------------------ adapters

@no_gpu
def test_lora_rejects(qmm_lib):
    K, M, r, L, N = 256, 70, 16, 5, 1100
    h = qmm_lib.lib()

    def call(a=None, b=None, x=None, base=None, y=None, ids=IDS, scales=WTS, ws=WS, size=1 << 24):
        return h.qmm_lora(*_ref(a or _adapters(K, r, L, W), b or _adapters(r, M, L, U), x or _dense(B.F32, K, N, X)), _v(ids), _v(scales),
                          *_ref(base, y or _dense(B.F32, M, N, Y)), _v(ws), size, None)

    def size(a, b, x):
        return h.qmm_lora_workspace_size(*_ref(a, b, x))

    a, b, x, y = _adapters(K, r, L, W), _adapters(r, M, L, U), _dense(B.F32, K, N, X), _dense(B.F32, M, N, Y)
    need = size(a, b, x)
    assert need > 0 and need % (N * 16 * 4) == 0 and need <= 4 * N * 16 * 4          # at most four parts of K
    assert size(a, b, _dense(B.F32, K, 1, X)) == size(a, b, _dense(B.F32, K, 0, 0)) == 0
    assert size(None, b, x) == size(a, None, x) == size(a, b, None) == size(a, _adapters(r, 0, L, 0), x) == 0
    for null in range(4):
        ds = [a, b, x, y]
        ds[null] = None
        assert h.qmm_lora(*_ref(*ds[:3]), _v(IDS), None, None, *_ref(ds[3]), _v(WS), 1 << 24, None) == B.ERR_NULL, null
    for t in (B.F32, B.F16):
        f = B.make_desc(t, K, r, 4 * K, W, n_dims=3)
        f.ne[2], f.nb[2] = L, 4 * K * r
        assert call(a=f) == B.ERR_TYPE
    assert call(a=B.make_desc(B.BF16, K, r, 2 * K, W)) == B.ERR_UNSUPPORTED
    assert call(x=_dense(B.F16, K, N, X)) == B.ERR_TYPE and call(y=_dense(B.BF16, M, N, Y)) == B.ERR_TYPE
    assert call(base=_dense(B.BF16, M, N, D)) == B.ERR_TYPE
    assert call(x=_dense(B.F32, K + 32, N, X)) == B.ERR_SHAPE
    assert call(a=_adapters(40, r, L, W), x=_dense(B.F32, 40, N, X)) == B.ERR_SHAPE
    for rank in (0, 4, 12, 136):
        assert call(a=_adapters(K, rank, L, W), b=_adapters(rank, M, L, U, pitch=288)) == B.ERR_SHAPE, rank
    assert call(b=_adapters(24, M, L, U)) == B.ERR_SHAPE and call(b=_adapters(r, M, L + 1, U)) == B.ERR_SHAPE
    assert call(a=_adapters(K, r, 0, W), b=_adapters(r, M, 0, U)) == B.ERR_SHAPE
    assert call(y=_dense(B.F32, M + 1, N, Y)) == B.ERR_SHAPE and call(y=_dense(B.F32, M, N + 1, Y)) == B.ERR_SHAPE
    assert call(base=_dense(B.F32, M, N - 1, D)) == B.ERR_SHAPE and call(base=_dense(B.F32, M + 4, N, D)) == B.ERR_SHAPE
    assert call(a=_adapters(K, r, L, W + 8)) == B.ERR_LAYOUT and call(a=_adapters(K, r, L, W, pitch=2 * K + 8)) == B.ERR_LAYOUT
    assert call(b=_adapters(r, M, L, U, apart=2 * r * M - 16)) == B.ERR_LAYOUT
    assert call(x=_dense(B.BF16, K, N, X + 8)) == B.ERR_LAYOUT and call(x=_dense(B.F32, K, N, X + 2)) == B.ERR_LAYOUT
    assert call(ids=0) == B.ERR_NULL and call(ws=0) == B.ERR_NULL
    assert call(ids=IDS + 1) == B.ERR_LAYOUT and call(scales=WTS + 2) == B.ERR_LAYOUT and call(ws=WS + 4) == B.ERR_LAYOUT
    assert call(size=need - 1) == B.ERR_SCRATCH
    assert call(ids=TOP) == B.ERR_UNSUPPORTED and call(scales=TOP) == B.ERR_UNSUPPORTED
    # operands that y or the workspace would change
    for at in (W, U + 64, X, IDS + 4 * N - 4, WTS, WS + need - 4):
        assert call(y=_dense(B.F32, M, N, at)) == B.ERR_ALIAS, hex(at)
    for at in (W, U, X, IDS, WTS):
        assert call(ws=at) == B.ERR_ALIAS, hex(at)
    assert call(base=_dense(B.F32, M, N, WS)) == B.ERR_ALIAS
    for base in (_dense(B.F32, M, N, Y + 4), _dense(B.F32, M, N, Y + 4 * M), _dense(B.F32, M, N, Y, pitch=4 * M + 4)):
        assert call(base=base) == B.ERR_ALIAS
    # pitches, tokens and outputs
    assert call(x=_dense(B.F32, K, 2, X, pitch=1 << 26), y=_dense(B.F32, M, 2, Y)) == B.ERR_UNSUPPORTED
    assert call(y=_dense(B.F32, M, N, Y, pitch=1 << 26)) == B.ERR_UNSUPPORTED
    assert call(base=_dense(B.F32, M, N, D, pitch=1 << 26)) == B.ERR_UNSUPPORTED
    assert call(a=_adapters(K, r, L, W, pitch=1 << 24)) == B.ERR_UNSUPPORTED
    assert call(b=_adapters(r, M, L, U, pitch=1 << 24)) == B.ERR_UNSUPPORTED
    n = (1 << 24) + 1
    assert call(x=_dense(B.F32, K, n, X), y=_dense(B.F32, M, n, Y)) == B.ERR_UNSUPPORTED
    m = 1 << 24
    assert call(b=_adapters(r, m, 1, U), a=_adapters(K, r, 1, W), y=_dense(B.F32, m, N, Y)) == B.ERR_UNSUPPORTED
    # nothing to do, and what is left to the GPU
    assert call(x=_dense(B.F32, K, 0, 0), y=_dense(B.F32, M, 0, 0), ids=0, ws=0, size=0) == B.OK
    assert call(b=_adapters(r, 0, L, 0), y=_dense(B.F32, 0, N, 0), ids=0, ws=0, size=0) == B.OK
    for base in (None, _dense(B.F32, M, N, D), y):
        assert call(base=base, size=need) == B.ERR_DEVICE
    assert call(scales=0) == B.ERR_DEVICE
    one = dict(x=_dense(B.F32, K, 1, X), y=_dense(B.F32, M, 1, Y), ws=0, size=0)
    assert call(**one) == B.ERR_DEVICE and call(**one, base=_dense(B.F32, M, 1, Y, pitch=4 * M + 64)) == B.ERR_DEVICE
