"""The layer of many tokens with h in two bf16 parts, in every form of its second
product (test_grouped_choice.py checks that the shapes take them), against a float64
reference: within the bounds of h rounded by 2^-16, and in norm, which tells it from h
in one part at any F."""
import numpy as np
import pytest
import torch

import grouped_ref as G
import quantized_matmul_ggml_amd as Q
from test_gpu_grouped import OUT, TYPES, _check, _dev, _layer, _x

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# experts, choices, tokens, F, M; by the form of the second product on a chip of 256 CUs
SHAPES = {"0": [(4, 2, 20, 320, 33), (4, 2, 20, 1024, 33), (4, 2, 20, 1600, 33), (64, 2, 50, 320, 2050)], "1": [(4, 2, 3000, 320, 600)],
          "2": [(4, 2, 1500, 320, 700)], "2deep": [(4, 2, 750, 1088, 530)], "4": [(4, 2, 700, 704, 400)], "4deep": [(4, 2, 600, 320, 270)]}
ALL = [pytest.param(*s, id="-".join([form, *map(str, s)])) for form, shapes in SHAPES.items() for s in shapes]
H_PARTS = 2.0 ** -16        # a part is off by half a step at most, 2^-8 of a value that is 2^-8 of h at most


def _reference(gate, up, down, x, ids, weights, bf16):
    """As grouped_ref.layer, with h off by H_PARTS, and twice the products in the second
    sum."""
    N, M, E = x.shape[0], down.shape[1], gate.shape[0]
    y, bound = np.zeros((N, M)), np.full((N, M), 1e-30)
    for e in range(E):
        n, s = np.nonzero(ids == e)
        if not n.size:
            continue
        h, eh = G.swiglu(*G.product(gate[e], x[n]), *G.product(up[e], x[n]))
        eh = eh + H_PARTS * (np.abs(h) + eh)
        d, ed = G.product(down[e], h)
        ed = 2 * ed + eh @ np.abs(down[e]).T * (1 + 2.0 ** -10)
        p = weights[n, s].astype(np.float64)[:, None]
        np.add.at(y, n, p * d)
        np.add.at(bound, n, np.abs(p) * (ed + (2 * ids.shape[1] + 2) * G.R.EPS * (np.abs(d) + ed)))
    return y, G.rounded(y, bound, bf16)


def _operands(kind, E, k, N, F, M, K=64, empty=True):
    rng = np.random.default_rng(E * F + N + M)
    ws, Ws = _layer(rng, kind, E, K, F, M)
    x, _ = _x(rng, N, K)
    x *= 0.125
    ids = np.stack([rng.permutation(E)[:k] for _ in range(N)]).astype(np.int32)
    w = rng.uniform(-0.2, 1, (N, k)).astype(np.float32)
    if empty:
        ids[rng.random(ids.shape) < 0.1] = -1
        w[ids < 0] = np.nan
    return ws, Ws, x, ids, w


def _split(ws, x, k):
    return torch.full((Q.moe_gemm_workspace_size(ws[0], ws[2], x, k, split=True),), 0xA5, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("kind", list(TYPES))
@pytest.mark.parametrize("E,k,N,F,M", ALL)
def test_layer(kind, E, k, N, F, M):
    print(f"[case] split layer {kind} E {E} k {k} N {N} F {F} M {M}", flush=True)
    ws, Ws, x, ids, w = _operands(kind, E, k, N, F, M)
    X = x.double().cpu().numpy()
    y = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), dtype=torch.bfloat16)
    ref, bound = _reference(*Ws, X, ids, w, True)
    _check(y, ref, bound, "bf16")
    ref, bound = _reference(*Ws, X, ids, w, False)
    z = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), workspace=_split(ws, x, k))
    _check(z, ref, bound, "f32")
    assert torch.equal(z.bfloat16(), y)
    # The bounds are of the worst case.  Terms of either sign leave the error's norm at
    # about h's own relative error: 2^-16 at most in two parts, and about 2^-8 / (2 sqrt 3)
    # in one, as the least workspace has it.
    norm = lambda v: np.linalg.norm(v.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert norm(z) < 2.0 ** -14
    need = Q.moe_gemm_workspace_size(ws[0], ws[2], x, k)
    one = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    assert norm(one) > 2.0 ** -11
    low = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), dtype=torch.bfloat16, workspace=torch.empty(need, dtype=torch.uint8, device=DEV))
    assert torch.equal(low, one.bfloat16())


def test_workspace_that_is_not_enough_for_two_parts():
    """A byte less is h in one part, and only what is used is written."""
    print("[case] split workspace", flush=True)
    ws, Ws, x, ids, w = _operands("q4_0", 4, 2, 60, 96, 40)
    need = Q.moe_gemm_workspace_size(ws[0], ws[2], x, 2)
    at = lambda size: torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    two = -(-4 * 120 * 96 // 256) * 256 - -(-2 * 120 * 96 // 256) * 256 + need
    assert need < two <= Q.moe_gemm_workspace_size(ws[0], ws[2], x, 2, split=True)
    outs = []
    for size in (need, two - 1, two, two + 256):
        space = at(size)
        outs.append(Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), workspace=space[:size]))
        assert (space[two if size >= two else need:] == 0xA5).all()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3]) and not torch.equal(outs[1], outs[2])


def test_special_values_stay_in_their_token():
    print("[case] split special values", flush=True)
    for kind in TYPES:
        ws, Ws, x, ids, w = _operands(kind, 4, 2, 300, 320, 70, empty=False)
        x[7, 3], x[150, 63], x[299] = float("nan"), float("inf"), 1e12       # the last one's h is about 1e25
        X = x.double().cpu().numpy()
        fine = np.setdiff1d(np.arange(300), [7, 150])
        ref, bound = _reference(*Ws, X[fine], ids[fine], w[fine], False)
        y = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), workspace=_split(ws, x, 2))
        assert torch.isnan(y[7]).all() and not torch.isfinite(y[150]).any()
        _check(y[fine], ref, bound, kind)


def test_replays():
    """The default of a bf16 y captured and replayed between eager calls."""
    print("[case] split replays", flush=True)
    ws, Ws, x, ids, w = _operands("mxfp4", 64, 8, 64, 128, 96)
    ids, w = _dev(ids), _dev(w)
    call = lambda: Q.moe_gemm_swiglu(*ws, x, ids, w, dtype=torch.bfloat16)
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call()
    for seed in range(3):
        x.copy_(torch.randn(x.shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed)) * 0.1)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()), f"seed {seed}"
        torch.cuda.synchronize()


def test_more_than_four_gigabytes_of_h():
    print("[case] split large", flush=True)
    E, k, N, F, M = 2, 1, 140001, 8192, 20
    ws, Ws, x, ids, w = _operands("mxfp4", E, k, N, F, M)
    y = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), dtype=torch.bfloat16)
    rows = np.array([0, 1, N // 2, N - 2, N - 1])
    ref, bound = _reference(*Ws, x[_dev(rows)].double().cpu().numpy(), ids[rows], w[rows], True)
    _check(y[_dev(rows)], ref, bound, "large")


def test_rows_too_long_for_two_parts():
    """From F = 2^22 on h has one part whatever the workspace has room for."""
    print("[case] split long", flush=True)
    ws, _, x, ids, w = _operands("mxfp4", 1, 1, 3, 1 << 22, 2, K=32, empty=False)
    y = Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w), dtype=torch.bfloat16)
    assert torch.equal(y, Q.moe_gemm_swiglu(*ws, x, _dev(ids), _dev(w)).bfloat16()) and torch.isfinite(y).all()
