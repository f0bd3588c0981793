"""The Python binding on the GPU: calls given a stream of their own while the
current stream is busy.  torch.cuda._sleep holds the current stream back for
some milliseconds, so that work which is wrongly put there comes too late."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 40_000_000           # clock cycles, some 20 ms


def _side():
    """A stream that has waited for all work so far."""
    torch.cuda.synchronize()
    return torch.cuda.Stream()


@pytest.mark.parametrize("layout", ["rows", "transposed", "gaps"])
@pytest.mark.parametrize("type_", [B.MXFP4, B.Q4_0, B.Q8_0])
def test_quantize_experts(type_, layout):
    print(f"[case] quantize_experts {type_} {layout}", flush=True)
    E, M, K = 5, 33, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    shape = {"rows": (E, M, K), "transposed": (E, K, M), "gaps": (E, M + 2, K)}[layout]
    w = torch.randn(shape, device=DEV, generator=g)
    w = {"rows": w, "transposed": w.transpose(1, 2), "gaps": w[:, :M]}[layout]
    want = [Q.quantize(w[e].contiguous(), type_).data for e in range(E)]
    assert torch.equal(Q.quantize_experts(w, type_).data, torch.stack(want))
    side = _side()
    torch.cuda._sleep(BUSY)
    q = Q.quantize_experts(w, type_, stream=side)
    junk = [torch.full((E * M, K), 7.0, device=DEV) for _ in range(3)]     # takes what the call may have given back
    side.synchronize()
    assert torch.equal(q.data, torch.stack(want))
    assert (q.type, q.K, q.M) == (type_, K, M) and torch.equal(q.expert(2).data, want[2])
    torch.cuda.synchronize()
    del junk


def test_quantize_experts_bf16():
    print("[case] quantize_experts bf16", flush=True)
    w = torch.randn((2, 64, 9), device=DEV).bfloat16().transpose(1, 2)
    q = Q.quantize_experts(w, B.MXFP4)
    rows = R.quantize_mxfp4(w.float().cpu().numpy().reshape(18, 64))
    assert np.array_equal(q.data.cpu().numpy().reshape(18, -1), rows)
