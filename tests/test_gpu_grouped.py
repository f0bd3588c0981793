"""Slots grouped by expert, products grouped by expert with ragged sizes, and the
mixture-of-experts layer for many tokens on the GPU, against float64 references
(tests/grouped_ref.py derives the bounds)."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"mxfp4": B.MXFP4, "q4_0": B.Q4_0, "q8_0": B.Q8_0, "q4_b64": B.Q4_B64, "q8_b64": B.Q8_B64}
OUT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---------------------------------------------------------------- grouping

@pytest.mark.parametrize("S,E", [(1, 1), (2, 1024), (63, 3), (64, 2), (65, 8), (1024, 1023), (1025, 1024), (4097, 128),
                                 (2048, 5), (2049, 5), (4096, 11), (8192, 7), (40000, 1024), (65536, 2), (65537, 2), (70000, 1),
                                 (131072, 9), (131073, 9), (200003, 300), (524288, 3), (600001, 64)])
def test_group(S, E):
    print(f"[case] group S {S} E {E}", flush=True)
    rng = np.random.default_rng(S + E)
    for name, ids in (("spread", rng.integers(0, E, S)), ("skewed", np.minimum(rng.geometric(0.2, S) - 1, E - 1)),
                      ("holes", rng.choice([-2 ** 31, -1, 0, E - 1, E, 2 ** 31 - 1], S)), ("none", np.full(S, -1))):
        ids = ids.astype(np.int32)
        offsets, order, place = Q.moe_group(_dev(ids), E)
        ro, rr, rp = G.group(ids, E)
        assert np.array_equal(offsets.cpu().numpy(), ro), name
        assert np.array_equal(order.cpu().numpy(), rr), name
        assert np.array_equal(place.cpu().numpy(), rp), name


def test_group_no_slots_and_shapes():
    print("[case] group S 0", flush=True)
    offsets, order, place = Q.moe_group(torch.empty((0, 2), dtype=torch.int32, device=DEV), 5)
    assert offsets.tolist() == [0] * 6 and order.numel() == 0 and place.shape == (0, 2)
    offsets, order, place = Q.moe_group(torch.tensor([[2, 0], [0, -1], [2, 2]], dtype=torch.int32, device=DEV), 3)
    assert offsets.tolist() == [0, 2, 2, 5] and order.tolist() == [1, 2, 0, 4, 5, 3]
    assert place.tolist() == [[2, 0], [1, -1], [3, 4]]


# ---------------------------------------------------------------- products

def _experts(rng, kind, E, M, K, pad=0):
    rows = R.random_rows(rng, kind, (E, M), K)
    data = torch.from_numpy(rows).to(DEV)
    if pad:
        wide = torch.full((E, M + 1, rows.shape[-1] + pad), 255, dtype=torch.uint8, device=DEV)
        wide[:, :M, :rows.shape[-1]] = data
        data = wide[:, :M]
    return Q.Experts(data, TYPES[kind], K, M), R.values(rows, kind, K)


def _x(rng, N, K, pad=0):
    """bf16 rows on the GPU (a pitch of K + pad elements, NaN between) and in float64."""
    x = torch.from_numpy((rng.standard_normal((N, K)) * 0.5 + 0.05).astype(np.float32)).bfloat16()
    wide = torch.full((N, K + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :K] = x.to(DEV)
    return wide[:, :K], x.double().numpy()


def _check(y, ref, bound, what):
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"{what}: worst {np.nanmax(err / bound)} of the bound"


# counts of rows per expert: tiles of 32, 64 and 128 rows, whole and cut
COUNTS = {"one": [1], "some": [25, 40, 0, 33], "few": [3, 0, 1, 33, 0, 2], "mid": [64, 0, 41, 130, 63], "many": [128, 5, 0, 300, 129],
          "ends": [0, 0, 257, 0]}


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("K,M", [(64, 1), (128, 130), (320, 70), (1088, 33), (4224, 40)])
def test_gemm_grouped(kind, counts, K, M):
    """Rows in order, tail rows outside all groups, then the same rows picked by an order."""
    n = COUNTS[counts]
    E, pad = len(n), 16 * (M % 2)
    if not kind.endswith("b64") and K == 320:
        K = 352                                     # an odd number of 32-blocks
    print(f"[case] grouped {kind} {counts} K {K} M {M}", flush=True)
    rng = np.random.default_rng(K * M + E)
    w, W = _experts(rng, kind, E, M, K, pad)
    up, U = _experts(rng, kind, E, M, K)
    tail, k = 3, 3
    total = sum(n) + tail
    offsets = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    x, X = _x(rng, total, K, pad // 2)
    slots = rng.permutation(total * k)[:total].astype(np.int32)
    for out in ("f32", "bf16"):
        for name, order, ws in (("rows", None, (w,)), ("picked", slots, (w,)), ("swiglu", slots, (w, up))):
            ref, bound, rows = G.grouped((W,) if len(ws) == 1 else (W, U), X, offsets, order, k, out == "bf16")
            y = torch.full((total, M + 5), 7.0, dtype=OUT[out], device=DEV)
            args = dict(order=None if order is None else _dev(order), top_k=k if order is not None else 1, out=y[:, :M])
            if len(ws) == 1:
                Q.gemm_grouped(w, x, _dev(offsets), **args)
            else:
                Q.gemm_grouped_swiglu(w, up, x, _dev(offsets), **args)
            _check(y[rows, :M], ref[rows], bound[rows], f"{name} {out}")
            rest = np.setdiff1d(np.arange(total), rows)
            assert (y[rest] == 7).all() and (y[:, M:] == 7).all(), f"{name} {out}: outside written"


@pytest.mark.parametrize("kind,E,n,K,M", [("mxfp4", 64, 5, 160, 40), ("q4_0", 200, 2, 96, 64), ("q8_0", 1024, 1, 64, 32),
                                          ("q4_b64", 65, 3, 64, 16), ("mxfp4", 40, 9, 2048, 530), ("q4_0", 48, 7, 1408, 600), ("q8_0", 3, 700, 64, 300), ("mxfp4", 2, 600, 4128, 140)])
def test_gemm_grouped_many(kind, E, n, K, M):
    """More experts than lanes, more tiles than XCDs, long rows."""
    print(f"[case] grouped {kind} E {E} rows {n} K {K} M {M}", flush=True)
    rng = np.random.default_rng(E + K)
    w, W = _experts(rng, kind, E, M, K)
    counts = rng.integers(0, 2 * n + 1, E)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, X = _x(rng, int(offsets[-1]), K)
    ref, bound, rows = G.grouped((W,), X, offsets, None, 1, False)
    y = Q.gemm_grouped(w, x, _dev(offsets))
    _check(y[rows], ref[rows], bound[rows], kind)


def test_gemm_grouped_wild_offsets_and_orders():
    """Offsets outside the rows are cut to them, tokens outside x count as zeros, rows
    of no group keep what they held: nothing outside is read or written."""
    print("[case] grouped wild offsets", flush=True)
    rng = np.random.default_rng(3)
    w, W = _experts(rng, "q4_0", 4, 48, 96)
    x, X = _x(rng, 20, 96)
    for offsets in ([-5, 4, 4, 9, 100], [0, 0, 0, 0, 0], [30, 40, 50, 60, 70], [-9, -8, -7, -6, -5], [2 ** 31 - 1] * 5,
                    [-2 ** 31, 0, 10, 20, 2 ** 31 - 1], [0, 15, 5, 20, 18]):
        y = torch.full((20, 48), 7.0, device=DEV)
        Q.gemm_grouped(w, x, torch.tensor(offsets, dtype=torch.int32, device=DEV), out=y)
        cut = np.clip(offsets, 0, 20)
        if (np.diff(cut) < 0).any():
            continue                                # whose rows then have which expert is not said
        ref, bound, rows = G.grouped((W,), X, cut, None, 1, False)
        _check(y[rows], ref[rows], bound[rows], str(offsets))
        assert (y[np.setdiff1d(np.arange(20), rows)] == 7).all()
    order = np.array([0, 39, 40, -1, -2, 2 ** 31 - 1, -2 ** 31, 1], np.int32)       # two slots a token: 20 tokens
    y = Q.gemm_grouped(w, x, torch.tensor([0, 2, 4, 6, 8], dtype=torch.int32, device=DEV), order=_dev(order), top_k=2)
    for r, (t, e) in enumerate(((0, 0), (19, 0), (None, 1), (None, 1), (None, 2), (None, 2), (None, 3), (0, 3))):
        if t is None:
            assert (y[r] == 0).all()
        else:
            ref, bound = G.product(W[e], X[t:t + 1])
            _check(y[r:r + 1], ref, bound, str(r))


@pytest.mark.parametrize("R", [4, 200])
def test_gemm_grouped_without_tokens(R):
    """Rows picked from an x without rows are zeros."""
    print(f"[case] grouped no tokens R {R}", flush=True)
    w, _ = _experts(np.random.default_rng(6), "q4_0", 2, 20, 64)
    y = Q.gemm_grouped(w, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV),
                       torch.tensor([0, R // 2, R], dtype=torch.int32, device=DEV),
                       order=torch.arange(R, dtype=torch.int32, device=DEV))
    assert y.shape == (R, 20) and (y == 0).all()


def test_gemm_grouped_special_values_stay_in_their_row():
    print("[case] grouped special values", flush=True)
    rng = np.random.default_rng(4)
    for kind in ("q4_0", "mxfp4", "q8_0"):
        w, W = _experts(rng, kind, 2, 40, 128)
        x, X = _x(rng, 50, 128)
        x[7, 3], x[30, 100], x[31, 5] = float("nan"), float("inf"), 1e38
        offsets = np.array([0, 20, 45], np.int32)
        ref, bound, rows = G.grouped((W,), X, offsets, None, 1, False)
        y = Q.gemm_grouped(w, x, _dev(offsets))
        assert torch.isnan(y[7]).all() and not torch.isfinite(y[30]).any()
        rest = np.setdiff1d(rows, [7, 30, 31])
        _check(y[rest], ref[rest], bound[rest], kind)


def test_mxfp4_not_a_number_block():
    print("[case] grouped mxfp4 NaN scale", flush=True)
    rng = np.random.default_rng(5)
    w, W = _experts(rng, "mxfp4", 1, 4, 96)
    w.data[0, 2, 1] = 255
    x, X = _x(rng, 3, 96)
    y = Q.gemm_grouped(w, x, torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    assert torch.isnan(y[:, 2]).all() and torch.isfinite(y[:, [0, 1, 3]]).all()


# ------------------------------------------------------------------- layer

def _layer(rng, kind, E, K, F, M, pad=0):
    parts = [_experts(rng, kind, E, m, c, pad) for m, c in ((F, K), (F, K), (M, F))]
    return [p[0] for p in parts], [p[1] for p in parts]


@pytest.mark.parametrize("kind,E,k,N,K,F,M", [("mxfp4", 8, 2, 1, 256, 96, 33), ("mxfp4", 32, 8, 70, 160, 64, 50),
                                              ("q4_0", 4, 2, 300, 288, 160, 130), ("q8_0", 5, 3, 40, 96, 352, 64),
                                              ("q4_b64", 6, 2, 129, 192, 128, 20), ("q8_b64", 3, 1, 200, 64, 64, 3)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_layer(kind, E, k, N, K, F, M, out):
    print(f"[case] layer {kind} E {E} k {k} N {N} K {K} F {F} M {M} {out}", flush=True)
    rng = np.random.default_rng(E * K + F + N)
    (g, u, d), (GW, UW, DW) = _layer(rng, kind, E, K, F, M, pad=16 * (N % 2))
    x, X = _x(rng, N, K, 8 * (N % 2))
    x *= 0.125
    X = x.double().cpu().numpy()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(N)]).astype(np.int32)
    ids[rng.random(ids.shape) < 0.1] = -1
    ids[rng.random(ids.shape) < 0.05] = E
    w = rng.uniform(-0.2, 1, (N, k)).astype(np.float32)
    w[(ids < 0) | (ids >= E)] = np.nan
    ref, bound = G.layer(GW, UW, DW, X, ids, w, out == "bf16")
    y = Q.moe_gemm_swiglu(g, u, d, x, _dev(ids), _dev(w), dtype=OUT[out])
    _check(y, ref, bound, kind)


def test_layer_repeated_and_empty():
    """Experts named twice by a token, tokens without experts, no tokens at all, and
    dimensions of zero."""
    print("[case] layer repeated", flush=True)
    rng = np.random.default_rng(8)
    (g, u, d), (GW, UW, DW) = _layer(rng, "q8_0", 3, 64, 96, 40)
    x, X = _x(rng, 5, 64)
    ids = np.array([[1, 1, 1], [-1, -1, -1], [2, 0, 2], [0, 3, 7], [1, 0, -1]], np.int32)
    w = rng.uniform(0, 1, (5, 3)).astype(np.float32)
    ref, bound = G.layer(GW, UW, DW, X, ids, w, False)
    y = Q.moe_gemm_swiglu(g, u, d, x, _dev(ids), _dev(w))
    _check(y, ref, bound, "repeated")
    assert (y[1] == 0).all()
    assert Q.moe_gemm_swiglu(g, u, d, x[:0], _dev(ids[:0]), _dev(w[:0])).shape == (0, 40)
    ex = lambda K, M: Q.Experts(torch.zeros((3, M, max(16, Q.row_size(Q.MXFP4, K))), dtype=torch.uint8, device=DEV), Q.MXFP4, K, M)
    for K, F, M in ((0, 32, 8), (64, 0, 8), (64, 32, 0)):
        print(f"[case] layer K {K} F {F} M {M}", flush=True)
        y = torch.full((5, M), 9.0, device=DEV)
        Q.moe_gemm_swiglu(ex(K, F), ex(K, F), ex(F, M), torch.ones((5, K), dtype=torch.bfloat16, device=DEV), _dev(ids), _dev(w), out=y)
        assert (y == 0).all()


def test_layer_is_its_parts():
    """The layer equals the calls it is made of, bit for bit."""
    print("[case] layer parts", flush=True)
    rng = np.random.default_rng(9)
    (g, u, d), _ = _layer(rng, "q4_0", 6, 128, 64, 72)
    x, _ = _x(rng, 90, 128)
    ids = _dev(rng.integers(-1, 6, (90, 2)).astype(np.int32))
    w = torch.rand((90, 2), device=DEV)
    offsets, order, place = Q.moe_group(ids, 6)
    h = Q.gemm_grouped_swiglu(g, u, x, offsets, order=order, top_k=2)
    p = Q.gemm_grouped(d, h, offsets)
    # the slots' sum in order, each step one fused multiply-add
    want = torch.zeros((90, 72), dtype=torch.float64, device=DEV)
    for s in range(2):
        live = (place[:, s] >= 0).unsqueeze(1)
        term = p[place[:, s].clamp(min=0).long()].double() * w[:, s].double().unsqueeze(1)
        want = torch.where(live, (want + term).float().double(), want)
    y = Q.moe_gemm_swiglu(g, u, d, x, ids, w)
    assert torch.equal(y.double(), want)


def test_layer_as_used_in_a_graph():
    """Router product, choice and layer of a prompt, captured and replayed: bit-equal
    to the eager calls."""
    rng = np.random.default_rng(11)
    E, k, K, F, N = 16, 4, 256, 96, 150
    for kind in ("mxfp4", "q8_0"):
        print(f"[case] prompt layer graph {kind}", flush=True)
        (g, u, d), (GW, UW, DW) = _layer(rng, kind, E, K, F, K)
        router = Q.f16_weight((torch.randn((E, K), device=DEV) * 0.05).half())
        x = torch.empty((N, K), dtype=torch.bfloat16, device=DEV)

        def step():
            ids, w = Q.moe_route(Q.gemm(router, x), k)
            return ids, w, Q.moe_gemm_swiglu(g, u, d, x, ids, w)

        x.copy_(torch.randn((N, K), device=DEV) * 0.1)
        step()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step()
        for seed in range(3):
            x.copy_(torch.randn((N, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) * 0.1)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            ref = step()
            torch.cuda.synchronize()
            for a, b in zip(outs, ref):
                assert torch.equal(a, b), f"seed {seed}"
            want, bound = G.layer(GW, UW, DW, x.double().cpu().numpy(), ref[0].cpu().numpy(), ref[1].cpu().numpy(), False)
            _check(outs[2], want, bound, f"seed {seed}")
