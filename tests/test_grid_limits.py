"""Sizes whose launches would have 2^32 threads or more along their grid, which
the runtime counts modulo 2^32 (it runs a part of the workgroups and reports
success): refused on the host.  Fake device addresses, so only where no GPU is
visible; the largest size that is not refused then ends at the launch."""
import ctypes

import pytest

from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.skipif(__import__("torch").cuda.device_count() > 0,
                                reason="fake device addresses: host-only validation checks run where no GPU is visible")

W, U, X, Y, D, IDS, WTS, WS = (0x100000000000 + (i << 40) for i in range(8))


def _ref(*ds):
    return [ctypes.byref(d) for d in ds]


def _experts(K, M, addr):
    t = B.make_desc(B.MXFP4, K, M, B.row_size(B.MXFP4, K), addr, n_dims=3)
    t.ne[2], t.nb[2] = 1, B.row_size(B.MXFP4, K) * M
    return t


def test_experts_output_rows(qmm_lib):
    """Eight rows per workgroup of 1024 threads: 2^25 - 8 rows at most, refused
    before the first of the two launches."""
    def call(M, K=32, F=32):
        g, u, d = _experts(K, F, W), _experts(K, F, U), _experts(F, M, D)
        x, y = B.make_desc(B.F32, K, 1, 4 * K, X), B.make_desc(B.F32, M, 1, 4 * M, Y)
        return qmm_lib.lib().qmm_moe_swiglu(*_ref(g, u, d, x), ctypes.c_void_p(IDS), ctypes.c_void_p(WTS), 1, *_ref(y),
                                            ctypes.c_void_p(WS), 1 << 30, None)

    for M in ((1 << 25) - 7, 1 << 25, (1 << 25) + 8, 1 << 28, (1 << 28) + 1):
        assert call(M) == B.ERR_UNSUPPORTED, M
    assert call((1 << 25) - 8) == B.ERR_DEVICE
    assert call(8, K=(1 << 28) + 32) == B.ERR_UNSUPPORTED and call(8, F=(1 << 28) + 32) == B.ERR_UNSUPPORTED


@pytest.mark.parametrize("kind", ["mxfp4 tokens", "mxfp4", "q4_0", "f16"])
def test_gemm_tiles(qmm_lib, kind):
    """512 threads per tile of 128 x 128 (fused pair: 64 rows): fewer than 2^23
    tiles, of one product or of a batch together."""
    K, type_ = 32, {"q4_0": B.Q4_0, "f16": B.F16}.get(kind, B.MXFP4)

    def weight(M, at=W):
        return B.make_desc(type_, K, M, B.row_size(type_, K), at)

    def tokens(N, at=X):
        return B.make_desc(B.MXFP4, K, N, 32, at) if kind == "mxfp4 tokens" else B.make_desc(B.BF16, K, N, 2 * K, at)

    def out(M, N, at=Y):
        return B.make_desc(B.F32, M, N, 4 * M, at)

    most = 1 << 30
    for M, N in ((1, most), (1, most - 127), (most, 1), (1 << 17, 1 << 20), (129, most >> 1), (1 << 33, 8), (8, 1 << 33)):
        assert B.call_raw("qmm_gemm", weight(M), tokens(N), out(M, N)) == B.ERR_UNSUPPORTED, (M, N)
    for M, N in ((1, most - 128), (most - 128, 1)):
        assert B.call_raw("qmm_gemm", weight(M), tokens(N), out(M, N)) == B.ERR_DEVICE, (M, N)
    if kind == "mxfp4 tokens":
        return
    for M, N in ((1, most), (most >> 1, 1), (65, most >> 1)):
        assert B.call_raw("qmm_gemm_swiglu", weight(M), weight(M, U), tokens(N), out(M, N)) == B.ERR_UNSUPPORTED, (M, N)
    assert B.call_raw("qmm_gemm_swiglu", weight((most >> 1) - 64), weight((most >> 1) - 64, U), tokens(1), out((most >> 1) - 64, 1)) == B.ERR_DEVICE

    def batch(*Ns):
        items = [B.QmmGemmItem(*(ctypes.pointer(d) for d in (weight(M, W + (i << 37)), tokens(1, X + (i << 37)), out(M, 1, Y + (i << 37)))))
                 for i, M in enumerate(Ns)]
        return qmm_lib.lib().qmm_gemm_batch((B.QmmGemmItem * len(items))(*items), len(items), None)

    assert batch(most >> 1, most >> 1) == B.ERR_UNSUPPORTED
    assert batch(most >> 1, (most >> 1) - 128) == B.ERR_DEVICE
