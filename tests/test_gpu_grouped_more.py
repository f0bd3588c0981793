"""Grouped products on the GPU against float64 references: many rows of few outputs."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q
from test_gpu_grouped import OUT, TYPES, _check, _dev, _experts, _x

pytestmark = pytest.mark.gpu

# pair, M, K, rows, experts
FEW_OUTPUTS = [(0, 33, 64, 30000, 8), (0, 70, 256, 20000, 3), (1, 17, 128, 25000, 8)]


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("shape", FEW_OUTPUTS, ids=lambda s: "-".join(map(str, s)))
def test_many_rows_of_few_outputs(kind, shape):
    pair, M, K, rows, E = shape
    print(f"[case] few outputs {kind} pair {pair} M {M} K {K} R {rows} E {E}", flush=True)
    rng = np.random.default_rng(rows + M)
    ws = [_experts(rng, kind, E, M, K) for _ in range(1 + pair)]
    offsets = np.concatenate([[0], np.cumsum(rng.multinomial(rows, rng.dirichlet(np.full(E, 0.7))))]).astype(np.int32)
    x, X = _x(rng, 700, K)
    order = rng.integers(0, 1400, rows).astype(np.int32)
    out = "bf16" if pair else "f32"
    ref, bound, live = G.grouped([w[1] for w in ws], X, offsets, order, 2, pair == 1)
    call = Q.gemm_grouped_swiglu if pair else Q.gemm_grouped
    y = call(*(w[0] for w in ws), x, _dev(offsets), order=_dev(order), top_k=2, dtype=OUT[out])
    _check(y[live], ref[live], bound[live], kind)
