"""Low-rank adapters of many requests beside a shared projection on the GPU,
against a float64 reference (tests/grouped_ref.py derives the bound)."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _bf16(rng, *shape):
    t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16()
    return t.to(DEV), t.double().numpy()


def _case(rng, N, L, r, K, M, kind):
    (a, A), (b, Bm) = _bf16(rng, L, r, K), _bf16(rng, L, M, r)
    x = torch.from_numpy((rng.standard_normal((N, K)) + 0.1).astype(np.float32))
    x = x.bfloat16() if kind == "bf16" else x
    ids = rng.integers(-1, L, N).astype(np.int32)
    s = rng.uniform(-2, 2, L).astype(np.float32)
    base = rng.standard_normal((N, M)).astype(np.float32)
    return a, A, b, Bm, x.to(DEV), x.double().numpy(), ids, s, base


def _check(y, ref, bound, what):
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bound).all(), f"{what}: worst {np.nanmax(err / bound)} of the bound"


@pytest.mark.parametrize("N,L,r,K,M", [(1, 1, 8, 32, 1), (1, 4, 16, 2048, 300), (2, 3, 24, 96, 33), (15, 40, 8, 160, 64),
                                       (16, 2, 32, 256, 31), (17, 5, 48, 288, 100), (33, 64, 64, 128, 130),
                                       (64, 24, 16, 4128, 70), (100, 3, 128, 544, 40), (300, 7, 40, 64, 257),
                                       (1500, 4, 16, 96, 48)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_lora(N, L, r, K, M, kind):
    print(f"[case] lora N {N} L {L} r {r} K {K} M {M} {kind}", flush=True)
    rng = np.random.default_rng(N * r + K + M)
    a, A, b, Bm, x, X, ids, s, base = _case(rng, N, L, r, K, M, kind)
    for scales, add in ((s, base), (None, None)):
        ref, bound = G.lora(A, Bm, X, ids, scales, add)
        y = Q.lora(a, b, x, _dev(ids), scales=None if scales is None else _dev(scales), base=None if add is None else _dev(add))
        _check(y, ref, bound, "scaled" if add is not None else "bare")
        none = ids < 0
        assert np.array_equal(y.cpu().numpy()[none], base[none] if add is not None else np.zeros_like(base[none]))


def test_lora_in_place_pitches_and_runs():
    """y the base itself, rows with gaps left as they are, prompts whose tokens stand
    together."""
    print("[case] lora in place", flush=True)
    rng = np.random.default_rng(1)
    N, L, r, K, M = 200, 5, 16, 128, 90
    a, A, b, Bm, x, X, ids, s, base = _case(rng, N, L, r, K, M, "f32")
    ids = np.sort(ids)
    wide_x = torch.full((N, K + 3), float("nan"), device=DEV)
    wide_x[:, :K] = x
    wide_a = torch.full((L, r + 1, K + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_a[:, :r, :K] = a
    wide_b = torch.full((L, M, r + 8), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide_b[:, :, :r] = b
    y = torch.full((N, M + 7), 7.0, device=DEV)
    y[:, :M] = _dev(base)
    Q.lora(wide_a[:, :r, :K], wide_b[:, :, :r], wide_x[:, :K], _dev(ids), scales=_dev(s), base=y[:, :M], out=y[:, :M])
    ref, bound = G.lora(A, Bm, X, ids, s, base)
    _check(y[:, :M], ref, bound, "in place")
    assert (y[:, M:] == 7).all()


@pytest.mark.parametrize("pad,shift", [(4, 0), (1, 0), (8, 3)])
def test_lora_many_tokens_at_any_alignment(pad, shift):
    """More than 512 binary32 tokens with aligned rows, odd pitches and odd starts."""
    print(f"[case] lora pad {pad} shift {shift}", flush=True)
    rng = np.random.default_rng(pad + shift)
    N, L, r, K, M = 530, 9, 16, 224, 40
    a, A, b, Bm, x, X, ids, s, base = _case(rng, N, L, r, K, M, "f32")
    ids = np.sort(ids)
    wide = torch.full((N, K + pad), float("nan"), device=DEV)
    view = wide[:, shift:shift + K]
    view.copy_(x)
    ref, bound = G.lora(A, Bm, X, ids, s, base)
    y = Q.lora(a, b, view, _dev(ids), scales=_dev(s), base=_dev(base))
    _check(y, ref, bound, "aligned" if pad % 4 == 0 and shift == 0 else "odd")


def test_lora_wild_ids_and_special_values_stay_in_their_token():
    print("[case] lora special values", flush=True)
    rng = np.random.default_rng(2)
    N, L, r, K, M = 40, 3, 16, 64, 50
    a, A, b, Bm, x, X, ids, s, base = _case(rng, N, L, r, K, M, "f32")
    ids = rng.choice([-2 ** 31, -1, 0, 2, 3, 2 ** 31 - 1], N).astype(np.int32)
    ids[[4, 5, 6]] = [0, 2, -1]
    b[1] = float("nan")                               # an adapter that nobody uses
    x[4, 3], x[6] = float("nan"), float("inf")
    base[9] = np.nan
    ref, bound = G.lora(A, Bm, X, ids, s, base)
    y = Q.lora(a, b, x, _dev(ids), scales=_dev(s), base=_dev(base))
    assert torch.isnan(y[4]).all() and torch.isnan(y[9]).all()
    rest = np.setdiff1d(np.arange(N), [4, 9])
    _check(y[rest], ref[rest], bound[rest], "others")


def test_lora_infinite_activation():
    print("[case] lora infinite x", flush=True)
    a = torch.zeros((1, 8, 32), dtype=torch.bfloat16, device=DEV)
    a[0, 0] = 1.0
    b = torch.ones((1, 4, 8), dtype=torch.bfloat16, device=DEV)
    b[0, :, 1:] = 0
    x = torch.ones((2, 32), device=DEV)
    x[0, 5] = float("inf")
    y = Q.lora(a, b, x, torch.zeros(2, dtype=torch.int32, device=DEV))
    # the other ranks' 0 * inf is not a number, as in the formula
    assert not torch.isfinite(y[0]).any() and (y[1] == 32).all()


def test_lora_empty():
    print("[case] lora empty", flush=True)
    mk = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(3, dtype=torch.int32, device=DEV)
    base = torch.ones((3, 5), device=DEV)
    assert torch.equal(Q.lora(mk(2, 8, 0), mk(2, 5, 8), torch.zeros((3, 0), device=DEV), ids, base=base), base)
    assert Q.lora(mk(2, 8, 32), mk(2, 5, 8), torch.zeros((0, 32), device=DEV), ids[:0]).shape == (0, 5)
    assert Q.lora(mk(2, 8, 32), mk(2, 0, 8), torch.zeros((3, 32), device=DEV), ids).shape == (3, 0)


def test_projection_with_adapters_in_a_graph():
    """The shared quantized projection and the adapters of its requests as a decode
    step runs them, captured and replayed: bit-equal to the eager calls."""
    rng = np.random.default_rng(3)
    N, L, r, K, M = 8, 6, 16, 256, 160
    a, A, b, Bm, x, X, ids, s, _ = _case(rng, N, L, r, K, M, "f32")
    w = Q.quantize(torch.randn((M, K), device=DEV) * 0.05, Q.Q4_0)
    W = Q.dequantize(w).double().cpu().numpy()
    ids_d, s_d = _dev(ids), _dev(s)
    print("[case] projection with adapters graph", flush=True)

    def step():
        y = Q.gemv(w, x)
        return Q.lora(a, b, x, ids_d, scales=s_d, base=y, out=y)

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for seed in range(3):
        x.copy_(torch.randn((N, K), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), f"seed {seed}"
        Xd = x.double().cpu().numpy()
        want, bound = G.lora(A, Bm, Xd, ids, s, Xd @ W.T)
        _check(out, want, bound + 1e-4 * (np.abs(Xd) @ np.abs(W).T) + 1e-6, f"seed {seed}")
