"""The workspace of a layer with h in two bf16 parts: its size, what of it is taken,
and what the binding allocates, on the CPU."""
import pytest
import torch

import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B
from test_grouped_abi import D, IDS, U, W, WS, WTS, X, Y, _dense, _ex, _ref, _v, no_gpu
from test_grouped_binding import _experts

K, F, M, E, N, k = 256, 128, 66, 8, 50, 2
up256 = lambda n: (n + 255) // 256 * 256


@no_gpu
@pytest.mark.parametrize("type_", [B.F32, B.BF16])
def test_all_of_the_workspace_is_checked(qmm_lib, type_):
    h = qmm_lib.lib()
    ops = [_ex(K, F, E, W), _ex(K, F, E, U), _ex(F, M, E, D), _dense(B.BF16, K, N, X)]
    need = h.qmm_moe_gemm_workspace_size(*_ref(ops[0], ops[2], ops[3]), k)
    two = need - up256(2 * N * k * F) + up256(4 * N * k * F)
    assert two <= need + 2 * N * k * F + 256

    def call(size, y=Y, ids=IDS, wts=WTS, ws=WS):
        return h.qmm_moe_gemm_swiglu(*_ref(*ops), _v(ids), _v(wts), k, *_ref(_dense(type_, M, N, y)), _v(ws), size, None)

    for size in (need, two - 1, two, two + 1, 1 << 40):
        assert call(size) == B.ERR_DEVICE, size          # past the checks: no GPU here
    assert call(need - 1) == B.ERR_SCRATCH
    # what lies behind the least workspace is an operand's, or h's
    for size, used in ((need, need), (two - 1, need), (two, two), (1 << 40, two)):
        for at in ({"y": WS + used - 256}, {"ids": WS + used - 256}, {"wts": WS + used - 256}):
            assert call(size, **at) == B.ERR_ALIAS, (size, at)
        for at in ({"y": WS + used}, {"ids": WS + used}, {"wts": WS + used}):
            assert call(size, **at) == B.ERR_DEVICE, (size, at)
    top = (1 << 64) - 256 - (two + 255) // 256 * 256
    assert call(two, ws=top + 512) == B.ERR_UNSUPPORTED


def test_what_the_binding_allocates(monkeypatch, qmm_lib):
    sizes = []
    monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
    monkeypatch.setattr(B, "_launch", lambda dev, stream, name, *args: sizes.append(args[-1]))
    g, d, x = _experts(K, F), _experts(F, M), torch.zeros((N, K), dtype=torch.bfloat16)
    ids, p = torch.zeros((N, k), dtype=torch.int32), torch.zeros((N, k))
    need, two = (Q.moe_gemm_workspace_size(g, d, x, k, split=s) for s in (False, True))
    assert 0 < need == Q.moe_gemm_workspace_size(g, d, x, k) and two == need + 2 * N * k * F + 256
    Q.moe_gemm_swiglu(g, g, d, x, ids, p)
    Q.moe_gemm_swiglu(g, g, d, x, ids, p, dtype=torch.bfloat16)
    Q.moe_gemm_swiglu(g, g, d, x, ids, p, out=torch.zeros((N, M), dtype=torch.bfloat16))
    Q.moe_gemm_swiglu(g, g, d, x, ids, p, workspace=torch.zeros(two, dtype=torch.uint8))
    assert sizes == [need, two, two, two]
    assert Q.moe_gemm_workspace_size(g, d, x[:0], k, split=True) == 0
    assert Q.moe_gemm_swiglu(g, g, d, x[:0], ids[:0], p[:0], dtype=torch.bfloat16).shape == (0, M) and sizes[-1] == 0
