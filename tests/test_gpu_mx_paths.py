"""The MXFP4 GEMV on every path that its launches can take: each kernel
instantiation in one pass and in several passes over K, with a tile group per
workgroup and with several, tokens divided or not, tiles split once more or not
(tests/test_row_plan.py checks that the list reaches all of them), against
float64.  Bounds as in test_gpu_mx.py."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROWS = 97               # different rows of a matrix, which repeats them

# (whether a gate / up pair, M, K, N)
PATHS = [
    (0, 20465, 32, 2), (0, 65557, 32, 2), (0, 1301, 1952, 6), (0, 20545, 160, 3), (0, 65997, 160, 4),
    (0, 635, 4928, 7), (0, 2307, 9504, 4), (0, 4659, 10048, 4), (0, 629, 4160, 5), (0, 2119, 4000, 7),
    (0, 2639, 2144, 4), (0, 4223, 4000, 7), (0, 11007, 4096, 5), (0, 11008, 4096, 4), (0, 65913, 960, 3),
    (0, 699, 6368, 5), (0, 2133, 9568, 3), (0, 4301, 9888, 3), (0, 1281, 4192, 2), (0, 2727, 2336, 8),
    (0, 2555, 4128, 1), (0, 32000, 4096, 8), (0, 4189, 8256, 4), (0, 32000, 4096, 2), (0, 16787, 4128, 3),
    (0, 629, 19424, 2), (0, 1357, 19552, 1), (0, 4457, 19232, 1), (0, 1, 32, 5), (0, 1, 32, 1), (0, 1, 4640, 7),
    (0, 1, 288, 4), (0, 1, 288, 1), (0, 2119, 3872, 6), (0, 16741, 800, 2), (0, 1, 9504, 3), (0, 1, 544, 7),
    (0, 2089, 2336, 8), (0, 1, 544, 1), (0, 1, 19008, 2), (0, 1, 19008, 1), (1, 1, 32, 3), (1, 1, 32, 1),
    (1, 32773, 32, 2), (1, 1, 160, 4), (1, 1, 160, 1), (1, 33181, 160, 1), (1, 1, 4768, 8), (1, 1057, 9920, 4),
    (1, 2091, 9760, 4), (1, 1, 288, 5), (1, 1033, 4064, 6), (1, 1, 288, 1), (1, 1069, 8128, 4), (1, 4615, 4032, 7),
    (1, 33319, 288, 2), (1, 32925, 928, 3), (1, 1, 6304, 5), (1, 1067, 9888, 3), (1, 2199, 10336, 3),
    (1, 1, 544, 2), (1, 1095, 2336, 8), (1, 1, 544, 1), (1, 1027, 8256, 3), (1, 2061, 8256, 4),
    (1, 16425, 1056, 2), (1, 32897, 1056, 3), (1, 1, 19104, 2), (1, 1, 19136, 1), (1, 2117, 19808, 1),
    (0, 2049, 32, 8), (0, 65545, 32, 6), (0, 4095, 11008, 8), (0, 4303, 4832, 7), (0, 2067, 160, 5),
    (0, 65669, 160, 7), (0, 8185, 5792, 8), (0, 8213, 4800, 7), (0, 2063, 288, 8), (0, 16407, 1056, 6),
    (0, 65559, 928, 8), (0, 16377, 7872, 8), (0, 8273, 6368, 6), (0, 65521, 704, 7), (0, 16753, 2080, 5),
    (0, 33467, 2080, 6), (0, 16379, 32864, 6), (0, 33001, 11008, 6), (1, 1025, 32, 8), (1, 32777, 32, 8),
    (1, 1063, 4768, 7), (1, 2077, 4768, 8), (1, 1031, 160, 7), (1, 33003, 160, 7), (1, 4093, 20416, 8),
    (1, 4293, 4768, 7), (1, 1029, 288, 5), (1, 4103, 2112, 8), (1, 32917, 928, 7), (1, 4089, 8544, 6),
    (1, 4191, 6336, 5), (1, 16377, 1440, 7), (1, 8413, 2112, 6), (1, 32789, 1056, 7), (1, 16377, 6464, 5),
    (1, 8369, 5184, 7), (0, 11008, 4096, 8), (0, 11007, 4096, 7), (0, 33001, 4096, 5), (0, 2047, 5632, 8),
    (0, 4095, 11008, 7),
]


def _matrix(rng, M, K):
    some = R.random_rows(rng, "mxfp4", (min(M, ROWS),), K)
    data = torch.from_numpy(some).to(DEV)[torch.arange(M, device=DEV) % len(some)]
    return B.Weight(data, B.MXFP4, K, M), R.values(some, "mxfp4", K)


@pytest.mark.parametrize("pair,M,K,N", PATHS)
def test_gemv_path(pair, M, K, N):
    """Every output against the reference, with pitches of the tokens and the
    outputs, and the bytes between the outputs left as they were."""
    print(f"[case] mxfp4 gemv path pair {pair} {M}x{K} N {N}", flush=True)
    rng = np.random.default_rng(M * 8 + K + N)
    g, G = _matrix(rng, M, K)
    wide = torch.from_numpy(rng.standard_normal((N, K + 5)).astype(np.float32)).to(DEV) * (0.1 if pair else 1.0)
    x = wide[:, 3:3 + K]
    xd = x.double().cpu().numpy()
    out = torch.full((N, M + 3), 7.0, device=DEV)
    y = out[:, 1:1 + M]
    gs, eg = xd @ G.T, (K + 64) * R.EPS * (np.abs(xd) @ np.abs(G).T)
    if pair:
        u, U = _matrix(rng, M, K)
        us, eu = xd @ U.T, (K + 64) * R.EPS * (np.abs(xd) @ np.abs(U).T)
        Q.gemv_swiglu(g, u, x, out=y)
        ref = R.swish(gs) * us
        lim = 1.1 * eg * (np.abs(us) + eu) + np.abs(R.swish(gs)) * eu + 2.0 ** -20 * np.abs(ref) + 1e-30
    else:
        Q.gemv(g, x, out=y)
        ref, lim = gs, eg + 1e-30
    o = out.cpu().numpy().astype(np.float64)
    assert (o[:, 0] == 7).all() and (o[:, 1 + M:] == 7).all()
    at = np.arange(M) % len(G)
    err = np.abs(o[:, 1:1 + M] - ref[:, at])
    assert (err <= lim[:, at]).all(), f"worst {np.nanmax(err / lim[:, at])} of the bound"
    again = torch.empty((N, M), device=DEV)
    Q.gemv_swiglu(g, u, x, out=again) if pair else Q.gemv(g, x, out=again)
    assert torch.equal(again, y)
