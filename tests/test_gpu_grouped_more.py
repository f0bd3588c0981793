"""Grouped products on the GPU against float64 references: many rows of few outputs,
and the most rows that one launch takes."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q
from test_gpu_grouped import OUT, TYPES, _check, _dev, _experts, _x

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

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


# pair, M, K, rows, experts, type: more tiles than a grid takes in the form estimated to be the fastest
MOST_ROWS = [(0, 16, 64, (1 << 27) + 33, 8, "mxfp4"), (1, 16, 2048, (1 << 28) + 77, 3, "q4_0")]


@pytest.mark.parametrize("shape", MOST_ROWS, ids=lambda s: "-".join(map(str, s)))
def test_most_rows(shape):
    """Every row against the table of all (expert, token) products."""
    pair, M, K, rows, E, kind = shape
    print(f"[case] most rows {shape}", flush=True)
    rng = np.random.default_rng(M + K)
    ws = [_experts(rng, kind, E, M, K) for _ in range(1 + pair)]
    x, X = _x(rng, 500, K)
    table, bound = [], []
    for e in range(E):
        v, b = G.product(ws[0][1][e], X)
        if pair:
            v, b = G.swiglu(v, b, *G.product(ws[1][1][e], X))
        table.append(v)
        bound.append(G.rounded(v, b, True))
    table, bound = (torch.from_numpy(np.concatenate(t)).to(DEV) for t in (table, bound))
    cuts = np.sort(rng.integers(0, rows, E - 1))
    offsets = _dev(np.concatenate([[0], cuts, [rows - 1]]).astype(np.int32))
    order = torch.randint(0, 500, (rows,), dtype=torch.int32, device=DEV)
    y = torch.full((rows, M), 7.0, dtype=torch.bfloat16, device=DEV)
    call = Q.gemm_grouped_swiglu if pair else Q.gemm_grouped
    call(*(w[0] for w in ws), x, offsets, order=order, out=y)
    assert (y[rows - 1] == 7).all()
    for at in range(0, rows - 1, 1 << 24):
        r = torch.arange(at, min(at + (1 << 24), rows - 1), device=DEV)
        pick = torch.searchsorted(offsets[1:].long(), r, right=True) * 500 + order[r].long()
        bad = (y[r].double() - table[pick]).abs() > bound[pick]
        assert not bad.any(), f"rows from {at} on"
