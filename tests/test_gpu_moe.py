"""The mixture-of-experts layer on the GPU: the router's choice, and the chosen
experts' SwiGLU blocks for 1 to 8 tokens, against float64 references
(tests/mx_ref.py derives the error bound)."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"mxfp4": B.MXFP4, "q4_0": B.Q4_0, "q8_0": B.Q8_0, "q4_b64": B.Q4_B64, "q8_b64": B.Q8_B64}


# ------------------------------------------------------------------ router

@pytest.mark.parametrize("N,E,k", [(1, 1, 1), (1, 8, 2), (5, 8, 8), (7, 60, 6), (3, 64, 16), (130, 65, 4), (33, 128, 8),
                                   (9, 256, 8), (4, 257, 5), (2, 1024, 16)])
def test_route(N, E, k):
    rng = np.random.default_rng(N * E + k)
    for masked in (False, True):
        l = (rng.standard_normal((N, E)) * 3).astype(np.float32)
        l[:, ::3] = np.round(l[:, ::3])                       # ties
        if masked:
            l[rng.random((N, E)) < 0.4] = -np.inf
            l[rng.random((N, E)) < 0.1] = np.nan
            l[0] = -np.inf                                    # nothing left
        for all_ in (True, False):
            print(f"[case] route N {N} E {E} k {k} masked {masked} all {all_}", flush=True)
            ids, w = Q.moe_route(torch.from_numpy(l).to(DEV), k, rule=Q.ROUTE_ALL if all_ else Q.ROUTE_CHOSEN)
            ri, rw = R.route(l, k, all_)
            assert np.array_equal(ids.cpu().numpy(), ri)
            # exp and its argument: a few ulps each of values up to e^0; the
            # sum of E terms adds (E / 64 + 6) roundings, the quotient one
            assert np.allclose(w.cpu().numpy(), rw, rtol=(E / 64 + 64) * R.EPS, atol=1e-38)


def test_route_ties_infinities_and_pitch():
    print("[case] route ties", flush=True)
    l = torch.zeros((3, 70), device=DEV)
    l[1, 5], l[1, 66] = np.inf, np.inf
    l[2] = -np.inf
    l[2, 69] = -1e30
    ids, w = Q.moe_route(l, 4, rule=Q.ROUTE_CHOSEN)
    assert ids.tolist() == [[0, 1, 2, 3], [5, 66, 0, 1], [69, -1, -1, -1]]
    assert w.tolist() == [[0.25] * 4, [0.5, 0.5, 0.0, 0.0], [1.0, 0.0, 0.0, 0.0]]
    big = torch.randn((6, 40), device=DEV)
    a, b = Q.moe_route(big[:, 3:20], 3), Q.moe_route(big[:, 3:20].contiguous(), 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert Q.moe_route(torch.empty((0, 8), device=DEV), 2)[0].shape == (0, 2)


# ----------------------------------------------------------------- experts

def _experts(rng, kind, E, M, K, pad=0):
    rows = R.random_rows(rng, kind, (E, M), K)
    data = torch.from_numpy(rows).to(DEV)
    if pad:
        wide = torch.full((E, M + 1, rows.shape[-1] + pad), 255, dtype=torch.uint8, device=DEV)
        wide[:, :M, :rows.shape[-1]] = data
        data = wide[:, :M]
    return Q.Experts(data, TYPES[kind], K, M), R.values(rows, kind, K)


def _layer(rng, kind, E, K, F, M, pad=0):
    parts = [_experts(rng, kind, E, m, c, pad) for m, c in ((F, K), (F, K), (M, F))]
    return [p[0] for p in parts], [p[1] for p in parts]


def _check(y, ref, bound, what):
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert (err <= bound).all(), f"{what}: worst {np.nanmax(err / bound)} of the bound"


SHAPES = [("mxfp4", 1, 1, 1, 32, 32, 1), ("mxfp4", 8, 2, 1, 2048, 544, 300), ("mxfp4", 16, 4, 8, 512, 256, 100),
          ("mxfp4", 4, 3, 5, 96, 160, 33), ("mxfp4", 40, 8, 8, 288, 96, 64), ("mxfp4", 3, 2, 3, 8192, 128, 17),
          ("mxfp4", 64, 16, 8, 128, 64, 48), ("mxfp4", 2, 2, 8, 4128, 64, 16),
          ("q4_0", 8, 2, 1, 2048, 544, 300), ("q4_0", 5, 3, 6, 96, 160, 33), ("q4_0", 40, 8, 8, 512, 64, 40),
          ("q4_0", 1, 1, 2, 32, 32, 1), ("q8_0", 8, 2, 2, 1024, 544, 130), ("q8_0", 5, 3, 7, 96, 160, 33),
          ("q8_0", 1, 1, 1, 32, 32, 16), ("q8_0", 12, 4, 8, 4128, 32, 20),
          ("q4_b64", 6, 2, 4, 320, 192, 50), ("q4_b64", 3, 2, 8, 2112, 64, 16), ("q8_b64", 6, 2, 5, 320, 192, 50),
          ("q8_b64", 2, 1, 1, 64, 64, 3)]


@pytest.mark.parametrize("kind,E,k,N,K,F,M", SHAPES)
def test_moe_swiglu(kind, E, k, N, K, F, M):
    print(f"[case] moe {kind} E {E} k {k} N {N} K {K} F {F} M {M}", flush=True)
    rng = np.random.default_rng(E * K + F + N)
    (g, u, d), (G, U, D) = _layer(rng, kind, E, K, F, M, pad=16 * (N % 2))
    x = (rng.standard_normal((N, K)) * 0.05 + 0.01).astype(np.float32)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(N)]).astype(np.int32)
    w = rng.uniform(-0.2, 1, (N, k)).astype(np.float32)
    ref, bound = R.moe(G, U, D, x.astype(np.float64), ids, w)
    y = Q.moe_swiglu(g, u, d, torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))
    _check(y, ref, bound, kind)


@pytest.mark.parametrize("kind,K", [("mxfp4", 2080), ("q4_0", 2080), ("q4_b64", 2112), ("q8_0", 1056), ("q8_b64", 1088)])
def test_moe_many_tiles(kind, K):
    """Enough tiles that a wave keeps eight units in flight, with rows that end
    inside the last ones, and experts with one to eight pairs."""
    E, k, N, F, M = 12, 6, 8, 704, 24
    print(f"[case] moe many tiles {kind} K {K}", flush=True)
    rng = np.random.default_rng(K)
    (g, u, d), (G, U, D) = _layer(rng, kind, E, K, F, M, pad=32)
    x = (rng.standard_normal((N, K)) * 0.05 + 0.01).astype(np.float32)
    ids = np.stack([np.concatenate([[0], 1 + rng.permutation(E - 1)[:k - 1]]) for _ in range(N)]).astype(np.int32)
    w = rng.uniform(-0.2, 1, (N, k)).astype(np.float32)
    ref, bound = R.moe(G, U, D, x.astype(np.float64), ids, w)
    y = Q.moe_swiglu(g, u, d, torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV))
    _check(y, ref, bound, kind)


@pytest.mark.parametrize("kind", ["mxfp4", "q4_0", "q8_0"])
def test_moe_empty_and_repeated_slots(kind):
    """Ids outside the range are empty slots (whatever their weight), a token
    without experts gets zeros, an expert named twice counts twice, all tokens
    may share one expert."""
    rng = np.random.default_rng(2)
    E, K, F, M, k, N = 6, 256, 192, 70, 4, 8
    (g, u, d), (G, U, D) = _layer(rng, kind, E, K, F, M)
    x = (rng.standard_normal((N, K)) * 0.1).astype(np.float32)
    cases = {
        "none": np.full((N, k), -1),
        "wild": rng.choice([-2 ** 31, -1, 0, 3, 5, 6, 7, 2 ** 31 - 1], (N, k)),
        "same": np.full((N, k), 2),
        "twice": np.array([[1, 4, 1, -1], [4, 4, 4, 1], [-1, 0, 0, 0], [5, -1, -1, 5], [1, 1, 4, 4], [2, 3, 2, 3],
                           [-1, -1, -1, 1], [0, 1, 2, 3]]),
    }
    for name, ids in cases.items():
        print(f"[case] moe {kind} slots {name}", flush=True)
        ids = ids.astype(np.int32)
        w = rng.uniform(0, 1, (N, k)).astype(np.float32)
        w[(ids < 0) | (ids >= E)] = np.nan
        ref, bound = R.moe(G, U, D, x.astype(np.float64), ids, w)
        out = torch.full((N, M), np.nan, device=DEV)
        Q.moe_swiglu(g, u, d, torch.from_numpy(x).to(DEV), torch.from_numpy(ids).to(DEV), torch.from_numpy(w).to(DEV), out=out)
        _check(out, ref, bound, name)
        if name == "none":
            assert (out == 0).all()


def test_moe_full_pairs():
    """8 tokens of 16 slots each, 128 pairs over 40 experts."""
    print("[case] moe 128 pairs", flush=True)
    rng = np.random.default_rng(6)
    (g, u, d), (G, U, D) = _layer(rng, "mxfp4", 40, 128, 96, 40)
    x = (rng.standard_normal((8, 128)) * 0.1).astype(np.float32)
    ids = np.stack([rng.permutation(40)[:16] for _ in range(8)]).astype(np.int32)
    ids[3, 2:9] = ids[3, 1]
    ids[7] = -1
    ids[7, 15] = 39
    w = rng.uniform(0, 1, (8, 16)).astype(np.float32)
    ref, bound = R.moe(G, U, D, x.astype(np.float64), ids, w)
    y = Q.moe_swiglu(g, u, d, *(torch.from_numpy(t).to(DEV) for t in (x, ids, w)))
    _check(y, ref, bound, "128 pairs")


def test_moe_special_values_stay_in_their_token():
    print("[case] moe special values", flush=True)
    rng = np.random.default_rng(7)
    (g, u, d), (G, U, D) = _layer(rng, "mxfp4", 4, 64, 64, 20)
    x = (rng.standard_normal((5, 64)) * 0.1).astype(np.float32)
    x[1, 3], x[3, 5] = np.nan, 1e30
    ids = np.array([[0, 1], [0, 1], [0, 1], [0, 2], [3, 0]], np.int32)
    w = np.full((5, 2), 0.5, np.float32)
    y = Q.moe_swiglu(g, u, d, *(torch.from_numpy(t).to(DEV) for t in (x, ids, w))).cpu()
    ref, bound = R.moe(G, U, D, x.astype(np.float64), ids, w)
    assert torch.isnan(y[1]).all()
    for n in (0, 2, 4):
        _check(y[n:n + 1], ref[n:n + 1], bound[n:n + 1], f"token {n}")


def test_moe_empty_dimensions():
    print("[case] moe empty dimensions", flush=True)
    ids, w = torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
    ex = lambda K, M: Q.Experts(torch.empty((3, M, max(16, Q.row_size(Q.MXFP4, K))), dtype=torch.uint8, device=DEV), Q.MXFP4, K, M)
    for K, F, M in ((0, 32, 8), (64, 0, 8), (64, 32, 0)):
        gate, down = ex(K, F), ex(F, M)
        gate.data.zero_(), down.data.zero_()
        y = torch.full((2, M), 9.0, device=DEV)
        Q.moe_swiglu(gate, gate, down, torch.ones((2, K), device=DEV), ids, w, out=y)
        assert (y == 0).all()
    y = Q.moe_swiglu(ex(64, 32), ex(64, 32), ex(32, 8), torch.empty((0, 64), device=DEV), ids[:0], w[:0])
    assert y.shape == (0, 8)


def test_layer_as_used_in_a_graph():
    """Router product, choice and experts as one decode step runs them, captured
    and replayed: bit-equal to the eager calls, right against float64."""
    rng = np.random.default_rng(11)
    E, k, K, F, N = 16, 4, 512, 288, 5
    for kind in ("mxfp4", "q8_0"):
        print(f"[case] moe layer graph {kind}", flush=True)
        (g, u, d), (G, U, D) = _layer(rng, kind, E, K, F, K)
        router = Q.f16_weight((torch.randn((E, K), device=DEV) * 0.05).half())
        x = torch.empty((N, K), device=DEV)

        def step():
            ids, w = Q.moe_route(Q.gemv(router, x), k)
            return ids, w, Q.moe_swiglu(g, u, d, x, ids, w)

        x.copy_(torch.randn((N, K), device=DEV))
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
            want, bound = R.moe(G, U, D, x.double().cpu().numpy(), ref[0].cpu().numpy(), ref[1].cpu().numpy())
            _check(outs[2], want, bound, f"seed {seed}")


def test_two_calls_with_their_own_workspaces():
    """Two layers on two streams at once, each with its own workspace."""
    print("[case] moe two streams", flush=True)
    rng = np.random.default_rng(12)
    (g, u, d), _ = _layer(rng, "q4_0", 8, 1024, 512, 256)
    xs = [torch.randn((8, 1024), device=DEV) * 0.1 for _ in range(2)]
    ids = torch.from_numpy(rng.integers(0, 8, (8, 4)).astype(np.int32)).to(DEV)
    w = torch.rand((8, 4), device=DEV)
    want = [Q.moe_swiglu(g, u, d, x, ids, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    wss = [torch.empty(Q.moe_workspace_size(g, x, 4), dtype=torch.uint8, device=DEV) for x in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = Q.moe_swiglu(g, u, d, xs[i], ids, w, workspace=wss[i])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_binding_refuses_mismatches():
    (g, u, d), _ = _layer(np.random.default_rng(0), "q4_0", 2, 64, 64, 8)
    x, ids, w = torch.zeros((2, 64), device=DEV), torch.zeros((2, 1), dtype=torch.int32, device=DEV), torch.ones((2, 1), device=DEV)
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x, ids.long(), w)
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x, ids[:1], w[:1])
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x, ids, w.cpu())
    with pytest.raises(Q.QmmError) as e:
        Q.moe_swiglu(g, u, d, x, ids, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == B.ERR_SCRATCH


def test_binding_refuses_other_types():
    (g, u, d), _ = _layer(np.random.default_rng(0), "q4_0", 2, 64, 64, 8)
    x, ids, w = torch.zeros((1, 64), device=DEV), torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV)
    with pytest.raises(ValueError):
        Q.moe_route(x.bfloat16(), 1)
    with pytest.raises(ValueError):
        Q.moe_route(x[0], 1)
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x.half(), ids, w)
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x, ids[0], w[0])
    with pytest.raises(ValueError):
        Q.moe_swiglu(g, u, d, x, ids, w, out=torch.empty((1, 8), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        Q.quantize(x.half(), Q.MXFP4)
