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
