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
