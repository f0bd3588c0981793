"""Sizes at the limits of what the mixture-of-experts entry points launch."""
import pytest
import torch

import quantized_matmul_ggml_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_route_more_tokens_than_one_grid():
    """A grid has fewer than 2^32 threads, 64 of them per token: 2^26 tokens and
    more are routed too."""
    N = (1 << 26) + 5
    print(f"[case] route N {N}", flush=True)
    l = torch.zeros((N, 2), device=DEV)
    l[::3, 1] = 1.0
    ids, w = Q.moe_route(l, 1, rule=Q.ROUTE_ALL)
    second = l[:, 1] > 0
    assert torch.equal(ids[:, 0], second.int())
    # e^-1 and its sum and quotient: a few roundings of 2^-24
    first, other = 0.5, 1.0 / (1.0 + 2.718281828459045 ** -1)
    want = torch.where(second, other, first)
    assert ((w[:, 0] - want).abs() <= 8 * 2.0 ** -24).all()


def test_experts_most_output_rows():
    """2^25 - 8 output rows, the most that one call takes: rows that repeat give
    results that repeat, to the last one, and equal those of a small layer."""
    M, F = (1 << 25) - 8, 32
    print(f"[case] moe M {M}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(1)
    up = Q.quantize_experts(torch.randn((1, F, 32), device=DEV, generator=g), Q.MXFP4)
    few = Q.quantize(torch.randn((128, F), device=DEV, generator=g), Q.MXFP4).data
    x, ids, p = torch.randn((1, 32), device=DEV, generator=g), torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    want = Q.moe_swiglu(up, up, Q.Experts(few.unsqueeze(0), Q.MXFP4, F, 128), x, ids, p)
    many = few.repeat(1 << 18, 1)[:M].unsqueeze(0)
    y = Q.moe_swiglu(up, up, Q.Experts(many, Q.MXFP4, F, M), x, ids, p)
    assert torch.equal(y, want.repeat(1, 1 << 18)[:, :M]) and (want != 0).any()
    with pytest.raises(Q.QmmError):
        Q.moe_swiglu(up, up, Q.Experts(few.repeat((1 << 18) + 1, 1).unsqueeze(0), Q.MXFP4, F, (1 << 25) + 8), x, ids, p)
