"""GEMM launches of the most tiles that one takes (fewer than 2^32 threads)."""
import pytest
import torch

import quantized_matmul_ggml_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_gemm_most_tokens():
    """2^23 - 1 tiles of one product, the most that one launch takes."""
    N, K, M = (1 << 30) - 128, 32, 2
    print(f"[case] mxfp4 gemm N {N}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    w = Q.quantize(torch.randn((M, K), device=DEV, generator=g), Q.MXFP4)
    few = Q.quantize(torch.randn((128, K), device=DEV, generator=g), Q.MXFP4)
    want = Q.gemm(w, few)
    many = Q.Weight(few.data.repeat((1 << 23) - 1, 1), Q.MXFP4, K, N)
    y = Q.gemm(w, many)
    assert (y.view(-1, 128, M) == want).all() and (want != 0).any()
