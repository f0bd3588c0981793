"""What the device arrays of grouped products may hold, in every form of launch
(test_grouped_choice.py checks that the shapes take them): offsets and orders that
point outside, an x without rows, infinities and NaN, blocks that are no number."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q
from test_gpu_grouped import OUT, TYPES, _check, _dev, _experts, _x

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 4
# pair, M, K, rows; by the form that they take on a chip of 256 CUs
SHAPES = {"0": [(0, 40, 192, 40), (1, 40, 192, 40)], "1": [(0, 600, 192, 5000), (1, 530, 192, 3000)],
          "2": [(0, 330, 192, 6000), (1, 330, 192, 3000)], "2deep": [(0, 330, 192, 1500), (1, 270, 192, 1000)],
          "4": [(0, 330, 1088, 1500), (1, 130, 1088, 2000)], "4deep": [(0, 130, 192, 300), (1, 70, 192, 300)]}
ALL = [pytest.param(*s, id=f"{form}-{'pair' if s[0] else 'one'}") for form, two in SHAPES.items() for s in two]


def _operands(kind, pair, M, K, seed):
    rng = np.random.default_rng(seed)
    ws = [_experts(rng, kind, E, M, K, 16 * i) for i in range(1 + pair)]
    return rng, [w[0] for w in ws], [w[1] for w in ws]


def _guarded(R, M, pair):
    """(rows R x M inside, all): with a row before and after and five columns beside."""
    y = torch.full((R + 2, M + 5), 7.0, dtype=OUT["bf16" if pair else "f32"], device=DEV)
    return y[1:-1, :M], y


def _call(ws, *args, **q):
    return (Q.gemm_grouped if len(ws) == 1 else Q.gemm_grouped_swiglu)(*ws, *args, **q)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pair,M,K,R", ALL)
def test_wild_offsets(kind, pair, M, K, R):
    """Cut to the rows that there are; rows of no group keep what they held."""
    print(f"[case] wild offsets {kind} pair {pair} M {M} K {K} R {R}", flush=True)
    rng, ws, Ws = _operands(kind, pair, M, K, R)
    x, X = _x(rng, R, K, 8)
    top = 2 ** 31 - 1
    for offsets in ([-5, R // 5, R // 5, R // 2 - 1, 5 * R], [0] * 5, [R] * 5, [R + 1, 2 * R, top, top, top], [-9, -8, -7, -6, -5], [top] * 5,
                    [-2 ** 31, 0, 1, R - 1, top], [-2 ** 31] * 4 + [top], [0, 3 * R // 4, R // 4, R, 9 * R // 10], [R, 0, R, 0, R]):
        y, whole = _guarded(R, M, pair)
        _call(ws, x, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=y)
        cut = np.clip(offsets, 0, R)
        if (np.diff(cut) >= 0).all():               # else it is not said which expert a row has
            ref, bound, rows = G.grouped(Ws, X, cut, None, 1, pair == 1)
            _check(y[rows], ref[rows], bound[rows], str(offsets))
            y[rows] = 7
            assert (y == 7).all(), f"{offsets}: rows outside all groups written"
        y.fill_(7)
        assert (whole == 7).all(), f"{offsets}: outside y written"


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pair,M,K,R", ALL)
def test_wild_orders(kind, pair, M, K, R):
    """Rows whose token is none of x's are zeros."""
    print(f"[case] wild orders {kind} pair {pair} M {M} K {K} R {R}", flush=True)
    rng, ws, Ws = _operands(kind, pair, M, K, R + 1)
    N, k = 50, 3
    x, X = _x(rng, N, K)
    order = rng.integers(0, N * k, R).astype(np.int32)
    bad = rng.random(R) < 0.3
    order[bad] = rng.choice([-1, -2, -k, -2 ** 31, N * k, N * k + 1, 2 ** 31 - 1], int(bad.sum()))
    offsets = np.array([0, R // 8, R // 8, R - R // 3, R], np.int32)
    ref, bound, rows = G.grouped(Ws, X, offsets, np.where(bad, 0, order), k, pair == 1)
    y, whole = _guarded(R, M, pair)
    _call(ws, x, _dev(offsets), order=_dev(order), top_k=k, out=y)
    assert rows.size == R and (y[_dev(bad)] == 0).all()
    good = np.flatnonzero(~bad)
    _check(y[good], ref[good], bound[good], kind)
    y.fill_(7)
    assert (whole == 7).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pair,M,K,R", ALL)
def test_without_tokens(kind, pair, M, K, R):
    """Rows picked from an x without rows are zeros."""
    print(f"[case] no tokens {kind} pair {pair} M {M} K {K} R {R}", flush=True)
    _, ws, _ = _operands(kind, pair, M, K, 6)
    y, whole = _guarded(R, M, pair)
    _call(ws, torch.empty((0, K), dtype=torch.bfloat16, device=DEV), torch.tensor([0, R // 2, R // 2, R - 1, R], dtype=torch.int32, device=DEV),
          order=torch.arange(R, dtype=torch.int32, device=DEV), out=y)
    assert (y == 0).all()
    y.fill_(7)
    assert (whole == 7).all()


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("pair,M,K,R", ALL)
def test_special_values_stay_in_their_row(kind, pair, M, K, R):
    print(f"[case] special values {kind} pair {pair} M {M} K {K} R {R}", flush=True)
    rng, ws, Ws = _operands(kind, pair, M, K, R + 2)
    x, X = _x(rng, R, K)
    nan, inf, huge = 7, R // 2, R - 2                       # in the first group, in two others' tiles, in the last one's
    x[nan, 3], x[inf, K - 1], x[huge, 5] = float("nan"), float("inf"), 1e38
    offsets = np.array([0, R // 3, R // 2 - 1, R - 5, R], np.int32)
    ref, bound, rows = G.grouped(Ws, X, offsets, None, 1, pair == 1)
    y = _call(ws, x, _dev(offsets), dtype=OUT["bf16" if pair else "f32"])
    assert torch.isnan(y[nan]).all() and not torch.isfinite(y[inf]).any()
    rest = np.setdiff1d(rows, [nan, inf, huge])
    _check(y[rest], ref[rest], bound[rest], kind)


@pytest.mark.parametrize("pair,M,K,R", ALL)
def test_mxfp4_not_a_number_block(pair, M, K, R):
    """A block of scale byte 255 reaches its expert's rows of its output, no others."""
    print(f"[case] NaN scale pair {pair} M {M} K {K} R {R}", flush=True)
    rng, ws, Ws = _operands("mxfp4", pair, M, K, R + 3)
    x, X = _x(rng, R, K)
    offsets = np.array([0, R // 3, R // 2, R - 5, R], np.int32)
    ref, bound, rows = G.grouped(Ws, X, offsets, None, 1, pair == 1)
    for w, e, m, block in zip(ws, (0, 2), (M - 1, 3), (K // 32 - 1, 0)):
        w.data[e, m, block] = 255
        ref[offsets[e]:offsets[e + 1], m] = np.nan
    y = _call(ws, x, _dev(offsets), dtype=OUT["bf16" if pair else "f32"])
    assert torch.equal(torch.isnan(y), torch.from_numpy(np.isnan(ref)).to(DEV))
    fine = ~np.isnan(ref)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err[fine] <= bound[fine]).all(), float((err[fine] / bound[fine]).max())
