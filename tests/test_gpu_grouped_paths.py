"""Every form that grouped products and adapters take on a chip of 256 CUs (tile
sizes, streamed rows, one launch or two, parts of K, shared tiles), with types
and layouts in turn; calls on other streams, two at once, and replayed."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import mx_ref as R
import quantized_matmul_ggml_amd as Q
from test_gpu_grouped import OUT, _check, _dev, _experts, _layer, _x
from test_gpu_lora import _case

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# pair, M, K, rows, experts
PRODUCTS = [(0, 600, 352, 6000, 8), (1, 400, 352, 6000, 8), (0, 400, 352, 6000, 8), (0, 400, 352, 4000, 8), (1, 270, 352, 4000, 8),
            (1, 200, 352, 4000, 8), (0, 130, 1056, 4000, 8), (0, 600, 352, 300, 8), (1, 130, 1056, 2000, 8), (1, 270, 352, 300, 8),
            (0, 270, 352, 700, 1), (0, 70, 2080, 150, 5), (1, 33, 2080, 70, 3), (0, 130, 5632, 300, 3), (0, 530, 1024, 64, 64),
            (0, 200, 96, 130, 64), (1, 129, 1024, 64, 64), (1, 65, 1056, 64, 64)]
# streamed rows with several tiles to a wave, whose types are said
STREAMED = [("mxfp4", 0, 2050, 128, 64, 64), ("q4_0", 0, 1030, 96, 256, 256), ("q4_b64", 1, 1030, 128, 64, 64), ("mxfp4", 1, 2050, 128, 64, 64),
            ("q8_0", 0, 1030, 512, 256, 256), ("q8_b64", 1, 1030, 512, 64, 64), ("q4_0", 1, 1030, 1024, 64, 64)]


def _product(kind, pair, M, K, rows, E, out):
    if kind.endswith("b64") or kind == "mxfp4":
        K = (K + 63) // 64 * 64
    print(f"[case] product {kind} pair {pair} M {M} K {K} R {rows} E {E} {out}", flush=True)
    rng = np.random.default_rng(M + K + rows)
    ws = [_experts(rng, kind, E, M, K) for _ in range(1 + pair)]
    counts = rng.multinomial(rows, rng.dirichlet(np.full(E, 0.7)))
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k = 2
    x, X = _x(rng, rows, K)
    order = rng.permutation(rows * k)[:rows].astype(np.int32)
    ref, bound, live = G.grouped([w[1] for w in ws], X, offsets, order, k, out == "bf16")
    call = Q.gemm_grouped_swiglu if pair else Q.gemm_grouped
    args = dict(order=_dev(order), top_k=k, dtype=OUT[out])
    y = call(*(w[0] for w in ws), x, _dev(offsets), **args)
    _check(y[live], ref[live], bound[live], kind)
    again = call(*(w[0] for w in ws), x, _dev(offsets), **args)
    assert torch.equal(y[live], again[live])                       # the order of the sums is fixed


@pytest.mark.parametrize("kind", ["mxfp4", "q4_0", "q8_0", "q4_b64", "q8_b64"])
@pytest.mark.parametrize("shape", PRODUCTS, ids=lambda s: "-".join(map(str, s)))
def test_products(kind, shape):
    _product(kind, *shape, "bf16" if shape[0] else "f32")


@pytest.mark.parametrize("shape", STREAMED, ids=lambda s: "-".join(map(str, s)))
def test_streamed(shape):
    _product(*shape, "f32" if shape[1] else "bf16")


# tokens, adapters, rank, K, M, activations, aligned rows of x
ADAPTERS = [(1, 1, 128, 512, 700, "f32", 1), (256, 9, 64, 64, 513, "bf16", 1), (3, 2, 8, 32, 1100, "bf16", 1), (70, 9, 32, 96, 2100, "f32", 0),
            (1000, 300, 16, 256, 1300, "f32", 0), (1, 2, 128, 1056, 33, "bf16", 1), (2, 2, 40, 2080, 33, "f32", 1), (3, 3, 16, 4128, 130, "f32", 0),
            (17, 20, 128, 1056, 33, "bf16", 1), (513, 4, 16, 4128, 33, "f32", 0), (600, 40, 24, 4128, 33, "f32", 0), (1500, 500, 16, 96, 33, "f32", 0),
            (4100, 3, 8, 32, 1000, "f32", 0), (513, 4, 16, 4128, 33, "bf16", 1), (513, 3, 128, 2080, 130, "f32", 1), (600, 100, 64, 4128, 65, "bf16", 1),
            (4100, 5, 24, 4128, 130, "f32", 1), (4100, 2, 16, 64, 2050, "bf16", 1), (4100, 3, 40, 32, 4100, "f32", 1), (1100, 2, 32, 1056, 2000, "f32", 1)]


@pytest.mark.parametrize("runs", [False, True], ids=["mixed", "prompts"])
@pytest.mark.parametrize("shape", ADAPTERS, ids=lambda s: "-".join(map(str, s)))
def test_adapters(shape, runs):
    N, L, r, K, M, kind, wide = shape
    print(f"[case] adapters N {N} L {L} r {r} K {K} M {M} {kind} wide {wide} runs {runs}", flush=True)
    rng = np.random.default_rng(N + r + K + M)
    a, A, b, Bm, x, X, ids, s, base = _case(rng, N, L, r, K, M, kind)
    if runs:
        ids = np.sort(ids)
    if not wide:                                      # rows that start between 16-byte units
        t = torch.zeros((N, K + 1), dtype=x.dtype, device=DEV)
        t[:, :K] = x
        x = t[:, :K]
    ref, bound = G.lora(A, Bm, X, ids, s, base)
    y = Q.lora(a, b, x, _dev(ids), scales=_dev(s), base=_dev(base))
    _check(y, ref, bound, "apart")
    z = _dev(base)
    assert Q.lora(a, b, x, _dev(ids), scales=_dev(s), base=z, out=z) is z and torch.equal(y, z)


# ------------------------------------------------------- streams and replays

BUSY = 40_000_000           # clock cycles, some 20 ms


def _calls(rng):
    """Calls with their own operands: one of each kind and form of workspace."""
    E, k, K, F, N, L, r = 12, 3, 256, 96, 150, 6, 128
    (g, u, d), _ = _layer(rng, "q4_0", E, K, F, K)
    x, _ = _x(rng, N, K)
    ids, w = _dev(rng.integers(-1, E, (N, k)).astype(np.int32)), torch.rand((N, k), device=DEV)
    many = _dev(rng.integers(-1, E, 70000).astype(np.int32))
    offsets, order, _ = Q.moe_group(ids, E)
    a, _, b, _, xf, _, aid, s, base = _case(rng, 1100, L, r, 1056, 300, "f32")
    aid, s, base = _dev(aid), _dev(s), _dev(base)
    return {"group": lambda **q: Q.moe_group(many, E, **q)[0],
            "products": lambda **q: Q.gemm_grouped_swiglu(g, u, x, offsets, order=order, top_k=k, out=torch.zeros((N * k, F), device=DEV), **q),
            "layer": lambda **q: Q.moe_gemm_swiglu(g, u, d, x, ids, w, **q),
            "one launch": lambda **q: Q.lora(a[:, :16, :256], b[:, :, :16], xf[:300, :256], aid[:300], scales=s, base=base[:300], **q),
            "few": lambda **q: Q.lora(a, b, xf[:30], aid[:30], scales=s, base=base[:30], **q),
            "prompt": lambda **q: Q.lora(a, b, xf, aid, scales=s, base=base, **q)}


def test_other_streams_and_two_at_once():
    """Calls on a stream of their own while the current one is held back, then two
    streams at once, each with its own workspace and outputs."""
    calls = _calls(np.random.default_rng(21))
    for name, call in calls.items():
        print(f"[case] side stream {name}", flush=True)
        want = call()
        torch.cuda.synchronize()
        one, two = torch.cuda.Stream(), torch.cuda.Stream()
        if name != "products":                        # whose output is made on the current stream
            torch.cuda._sleep(BUSY)
            y = call(stream=one)
            junk = [torch.full((1 << 20,), 7.0, device=DEV) for _ in range(3)]
            one.synchronize()
            assert torch.equal(y, want), name
            torch.cuda.synchronize()
            del junk
        outs = []
        for i in range(6):
            with torch.cuda.stream((one, two)[i % 2]):
                outs.append(call())
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in outs), name


def test_replays():
    """Captured, replayed several times between eager calls: every replay equals them.
    Two graphs with workspaces of their own, replayed on two streams at once."""
    for name, call in _calls(np.random.default_rng(22)).items():
        print(f"[case] replay {name}", flush=True)
        want = call().clone()
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                out = call()
            graphs.append((graph, out, side))
        for _ in range(3):
            for graph, out, side in graphs:
                out.zero_()
            torch.cuda.synchronize()
            for graph, out, side in graphs:
                with torch.cuda.stream(side):
                    graph.replay()
            torch.cuda.synchronize()
            for graph, out, side in graphs:
                assert torch.equal(out, want), name
            assert torch.equal(call(), want)
            torch.cuda.synchronize()


def test_given_workspaces():
    """Workspaces with bytes beyond their size, which keep what they held."""
    print("[case] given workspaces", flush=True)
    rng = np.random.default_rng(23)
    E, k, K, F, N = 9, 2, 128, 64, 130
    (g, u, d), _ = _layer(rng, "mxfp4", E, K, F, 40)
    x, _ = _x(rng, N, K)
    ids, w = _dev(rng.integers(-1, E, (N, k)).astype(np.int32)), torch.rand((N, k), device=DEV)
    a, _, b, _, xf, _, aid, s, base = _case(rng, 1030, 5, 24, 64, 70, "bf16")
    many = _dev(rng.integers(0, E, 66000).astype(np.int32))
    for name, need, call in (("layer", Q.moe_gemm_workspace_size(g, d, x, k), lambda ws: Q.moe_gemm_swiglu(g, u, d, x, ids, w, workspace=ws)),
                             ("lora", Q.lora_workspace_size(a, b, xf), lambda ws: Q.lora(a, b, xf, _dev(aid), scales=_dev(s), workspace=ws)),
                             ("group", Q.moe_group_workspace_size(66000, E), lambda ws: Q.moe_group(many, E, workspace=ws)[1])):
        ws = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        assert need > 0 and torch.equal(call(ws[:need]), call(None)), name
        assert (ws[need:] == 0xA5).all(), name
        with pytest.raises(Q.QmmError):
            call(ws[:need - 16])


# ------------------------------------------------------ beyond 32-bit offsets

def _rows_of(w, W_of, x, y, rows, expert_of, what):
    """Rows of y against float64 products of a few experts, dequantized one at a time."""
    for r in rows:
        ref, bound = G.product(W_of(expert_of(r)), x[r:r + 1].double().cpu().numpy())
        _check(y[r:r + 1], ref, bound, f"{what} row {r}")


@pytest.mark.parametrize("K,M,R", [(8192, 40, 270001), (64, 8200, 140001)], ids=["x", "y"])
def test_more_than_four_gigabytes_of_rows(K, M, R):
    print(f"[case] large rows K {K} M {M} R {R}", flush=True)
    rng = np.random.default_rng(K)
    w, W = _experts(rng, "q8_0", 2, M, K)
    x = torch.randn((R, K), device=DEV, dtype=torch.bfloat16)
    cut = R - 77
    y = Q.gemm_grouped(w, x, torch.tensor([0, cut, R], dtype=torch.int32, device=DEV))
    _rows_of(w, lambda e: W[e], x, y, [0, 1, R // 2, cut - 1, cut, R - 1], lambda r: int(r >= cut), "large")
    if K == 64:                                            # picked rows read x from its start
        order = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV)
        z = Q.gemm_grouped(w, x, torch.tensor([0, R, R], dtype=torch.int32, device=DEV), order=order)
        for r in (0, R // 2, R - 1):
            ref, bound = G.product(W[0], x[R - 1 - r:R - r].double().cpu().numpy())
            _check(z[r:r + 1], ref, bound, f"picked row {r}")


@pytest.mark.parametrize("rows", [1, 40], ids=["streamed", "tiles"])
def test_more_than_four_gigabytes_of_experts(rows):
    E, M, K = 1024, 1040, 8192
    print(f"[case] large experts rows {rows}", flush=True)
    data = torch.randint(0, 256, (E, M, Q.row_size(Q.MXFP4, K)), dtype=torch.uint8, device=DEV)
    data[:, :, :K // 32] = torch.randint(118, 124, (E, M, K // 32), dtype=torch.uint8, device=DEV)
    assert data.numel() > 1 << 32
    w = Q.Experts(data, Q.MXFP4, K, M)
    counts = torch.full((E,), rows, dtype=torch.int32, device=DEV)
    counts[::3] = 0
    offsets = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), counts.cumsum(0).int()])
    n = int(offsets[-1])
    x = torch.randn((n, K), device=DEV, dtype=torch.bfloat16)
    y = Q.gemm_grouped(w, x, offsets)
    owner = torch.repeat_interleave(torch.arange(E, device=DEV), counts.long()).cpu().numpy()
    _rows_of(w, lambda e: R.values(data[e].cpu().numpy(), "mxfp4", K), x, y, [0, n // 2, n - 1], lambda r: int(owner[r]), "experts")


def test_more_than_four_gigabytes_of_outputs_of_adapters():
    N, M, K, r, L = 140001, 8200, 32, 16, 3
    print("[case] large adapters", flush=True)
    rng = np.random.default_rng(31)
    a, A, b, Bm, x, X, ids, s, _ = _case(rng, N, L, r, K, 4, "bf16")
    b = torch.randn((L, M, r), device=DEV).bfloat16()
    base = torch.full((N, M), 0.5, device=DEV)
    y = Q.lora(a, b, x, _dev(ids), scales=_dev(s), base=base, out=base)
    for n in (0, N // 2, N - 2, N - 1):
        ref, bound = G.lora(A, b.double().cpu().numpy(), X[n:n + 1], ids[n:n + 1], s, np.full((1, M), 0.5, np.float32))
        _check(y[n:n + 1], ref, bound, f"token {n}")
