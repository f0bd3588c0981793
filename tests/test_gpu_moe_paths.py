"""The experts on every path that their launches can take (depths, one and
several passes over K; tests/test_row_plan.py checks the list), with wide
outputs, pitches of the tokens and the outputs, and on a stream of their own."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from test_gpu_moe import TYPES, _check, _layer

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (type, E, k, N, K, F, M)
PATHS = [
    # several passes over K of an image for two pairs, and of one for one pair too
    ("mxfp4", 4, 4, 8, 4128, 544, 40), ("mxfp4", 4, 3, 7, 5664, 544, 24), ("q4_0", 4, 4, 8, 4128, 544, 40),
    ("q4_0", 4, 3, 7, 5664, 544, 24), ("q8_0", 4, 4, 8, 2816, 544, 40), ("q8_0", 4, 3, 7, 5664, 544, 24),
    ("q4_b64", 4, 4, 8, 4160, 576, 40), ("q8_b64", 4, 4, 8, 2880, 576, 40), ("mxfp4", 1, 1, 1, 22016, 96, 9),
    ("q8_0", 2, 2, 1, 22048, 96, 9), ("mxfp4", 3, 2, 3, 22016, 96, 33),
    # depths of two, four and eight units, one pass
    ("mxfp4", 6, 3, 8, 160, 800, 70), ("mxfp4", 6, 3, 8, 1056, 800, 70), ("mxfp4", 6, 3, 8, 2080, 800, 70),
    ("q4_0", 6, 3, 8, 160, 800, 70), ("q4_0", 6, 3, 8, 1056, 800, 70), ("q4_0", 6, 3, 8, 2080, 800, 70),
    ("q8_0", 6, 3, 8, 96, 800, 70), ("q8_0", 6, 3, 8, 544, 800, 70), ("q8_0", 6, 3, 8, 1120, 800, 70),
    ("mxfp4", 6, 3, 8, 416, 800, 70), ("q4_0", 6, 3, 8, 416, 800, 70), ("q8_0", 6, 3, 8, 224, 800, 70),
    # wide outputs
    ("mxfp4", 3, 2, 5, 256, 160, 2049), ("q4_0", 3, 2, 3, 256, 160, 4100), ("q8_0", 3, 2, 8, 256, 160, 777),
    ("q4_b64", 3, 2, 2, 256, 192, 1031), ("q8_b64", 3, 2, 6, 256, 192, 1500),
]


@pytest.mark.parametrize("kind,E,k,N,K,F,M", PATHS)
def test_moe_path(kind, E, k, N, K, F, M):
    print(f"[case] moe path {kind} E {E} k {k} N {N} K {K} F {F} M {M}", flush=True)
    rng = np.random.default_rng(E * K + F + N + M)
    (g, u, d), (G, U, D) = _layer(rng, kind, E, K, F, M, pad=16)
    wide = torch.from_numpy((rng.standard_normal((N, K + 7)) * 0.05 + 0.01).astype(np.float32)).to(DEV)
    x = wide[:, 3:3 + K]
    ids = np.stack([rng.permutation(E)[:k] for _ in range(N)]).astype(np.int32)
    w = rng.uniform(-0.2, 1, (N, k)).astype(np.float32)
    ref, bound = R.moe(G, U, D, x.double().cpu().numpy(), ids, w)
    out = torch.full((N, M + 6), 7.0, device=DEV)
    y, ids, w = out[:, 5:5 + M], torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV)
    Q.moe_swiglu(g, u, d, x, ids, w, out=y)
    _check(y, ref, bound, kind)
    o = out.cpu().numpy()
    assert (o[:, :5] == 7).all() and (o[:, 5 + M:] == 7).all()
    # on a stream of its own, with a workspace that it makes there, and packed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = Q.moe_swiglu(g, u, d, x.contiguous(), ids, w, stream=side)
    side.synchronize()
    assert torch.equal(again, y)
