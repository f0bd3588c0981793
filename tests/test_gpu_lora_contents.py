"""What the device arrays of low-rank adapters may hold, in every form of launch
(test_grouped_choice.py checks that the shapes take them): ids of no adapter,
infinities and NaN in tokens, adapters, scales and base."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q
from test_gpu_lora import _case, _check, _dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# tokens, adapters, rank, K, M; by the form that they take on a chip of 256 CUs
SHAPES = {"one launch": (40, 4, 16, 64, 50), "registers": (300, 4, 64, 1120, 70), "tiles": (1100, 4, 24, 96, 130)}


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("runs", [False, True], ids=["mixed", "prompts"])
@pytest.mark.parametrize("form", list(SHAPES))
def test_special_values_stay_in_their_token(form, runs, kind):
    N, L, r, K, M = SHAPES[form]
    print(f"[case] adapters' contents {form} runs {runs} {kind}", flush=True)
    rng = np.random.default_rng(N + K)
    a, A, b, Bm, x, X, _, s, base = _case(rng, N, L, r, K, M, kind)
    ids = rng.choice([-2 ** 31, -7, -1, 0, 1, 2, L, L + 1, 2 ** 31 - 1], N).astype(np.int32)
    if runs:
        ids = np.sort(ids)
    none = (ids < 0) | (ids >= L)
    lost = np.zeros(N, bool)                             # tokens without a value to compare with
    some, other = np.flatnonzero(~none), np.flatnonzero(none)
    x[int(some[0]), 3], x[int(some[-1]), K - 1] = float("nan"), float("-inf")
    lost[[some[0], some[-1]]] = True
    x[int(other[0])], x[int(other[-1])] = float("inf"), float("nan")
    base[some[1], M - 1] = np.nan
    b[3], s[3] = float("nan"), np.nan                    # an adapter that nobody uses
    a[2, r - 1, K - 1] = float("nan")                    # one that some tokens use
    lost |= ids == 2
    b[1, M // 2, 0] = float("inf")                       # one output of one adapter's tokens
    A, Bm = np.nan_to_num(A, posinf=0), np.nan_to_num(Bm, posinf=0)
    with np.errstate(invalid="ignore"):
        ref, bound = G.lora(A, Bm, np.where(np.isfinite(X), X, 0), np.where(none, -1, ids), np.nan_to_num(s), base)
    y = Q.lora(a, b, x, _dev(ids), scales=_dev(s), base=_dev(base))
    got = y.double().cpu().numpy()
    assert np.array_equal(y.cpu().numpy()[none], base[none])
    assert np.isnan(got[some[0]]).all() and not np.isfinite(got[some[-1]]).any() and np.isnan(got[ids == 2]).all()
    assert not np.isfinite(got[ids == 1][:, M // 2]).any()
    assert np.isnan(got[some[1], M - 1])
    keep = np.ones((N, M), bool)
    keep[lost] = False
    keep[ids == 1, M // 2] = False
    keep[some[1], M - 1] = False
    err = np.abs(got - ref)
    assert (err[keep] <= bound[keep]).all(), float(np.nanmax(err[keep] / bound[keep]))
