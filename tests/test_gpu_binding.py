"""The Python binding on the GPU: calls given a stream of their own while the
current stream is busy.  torch.cuda._sleep holds the current stream back for
some milliseconds, so that work which is wrongly put there comes too late."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 40_000_000           # clock cycles, some 20 ms


def _side():
    """A stream that has waited for all work so far."""
    torch.cuda.synchronize()
    return torch.cuda.Stream()


@pytest.mark.parametrize("layout", ["rows", "transposed", "gaps"])
@pytest.mark.parametrize("type_", [B.MXFP4, B.Q4_0, B.Q8_0])
def test_quantize_experts(type_, layout):
    print(f"[case] quantize_experts {type_} {layout}", flush=True)
    E, M, K = 5, 33, 96
    g = torch.Generator(device=DEV).manual_seed(3)
    shape = {"rows": (E, M, K), "transposed": (E, K, M), "gaps": (E, M + 2, K)}[layout]
    w = torch.randn(shape, device=DEV, generator=g)
    w = {"rows": w, "transposed": w.transpose(1, 2), "gaps": w[:, :M]}[layout]
    want = [Q.quantize(w[e].contiguous(), type_).data for e in range(E)]
    assert torch.equal(Q.quantize_experts(w, type_).data, torch.stack(want))
    side = _side()
    torch.cuda._sleep(BUSY)
    q = Q.quantize_experts(w, type_, stream=side)
    junk = [torch.full((E * M, K), 7.0, device=DEV) for _ in range(3)]     # takes what the call may have given back
    side.synchronize()
    assert torch.equal(q.data, torch.stack(want))
    assert (q.type, q.K, q.M) == (type_, K, M) and torch.equal(q.expert(2).data, want[2])
    torch.cuda.synchronize()
    del junk


def test_quantize_experts_bf16():
    print("[case] quantize_experts bf16", flush=True)
    w = torch.randn((2, 64, 9), device=DEV).bfloat16().transpose(1, 2)
    q = Q.quantize_experts(w, B.MXFP4)
    rows = R.quantize_mxfp4(w.float().cpu().numpy().reshape(18, 64))
    assert np.array_equal(q.data.cpu().numpy().reshape(18, -1), rows)


def test_calls_on_a_busy_streams_side():
    """With the current stream held back, memory that it has freed but not yet
    written to must not become a side call's output or workspace: what is
    pending there would write over it."""
    K, M, N, E, k = 1024, 512, 6, 4, 2
    g = torch.Generator(device=DEV).manual_seed(5)
    w = Q.quantize(torch.randn((M, K), device=DEV, generator=g) * 0.05, B.Q4_0)
    mx = Q.quantize(torch.randn((M, K), device=DEV, generator=g) * 0.05, B.MXFP4)
    up = Q.quantize_experts(torch.randn((E, M, K), device=DEV, generator=g) * 0.05, B.MXFP4)
    down = Q.quantize_experts(torch.randn((E, K, M), device=DEV, generator=g) * 0.05, B.MXFP4)
    x = torch.randn((N, K), device=DEV, generator=g)
    xb, xl = x.bfloat16(), torch.randn((N, E), device=DEV, generator=g)
    ids, p = Q.moe_route(xl, k)
    rec = Q.rows_to_records(w)
    calls = {
        "quantize": lambda s: Q.quantize(x, B.Q8_0, pitch=Q.row_size(B.Q8_0, K) + 32, stream=s).data,
        "dequantize": lambda s: Q.dequantize(mx, stream=s), "gemv": lambda s: Q.gemv(mx, x, stream=s),
        "gemv_swiglu": lambda s: Q.gemv_swiglu(w, w, x, stream=s), "gemm": lambda s: Q.gemm(w, xb, stream=s),
        "gemm_swiglu": lambda s: Q.gemm_swiglu(w, w, xb, stream=s), "gemm_batch": lambda s: Q.gemm_batch([(w, xb, None)], stream=s)[0],
        "gemv_batch": lambda s: Q.gemv_batch([(w, x, None)], stream=s)[0],
        "records_to_rows": lambda s: Q.records_to_rows(rec, B.Q4_0, K, M, pitch=w.pitch + 16, stream=s).data,
        "rows_to_records": lambda s: Q.rows_to_records(w, stream=s),
        "moe_route": lambda s: torch.cat([t.float() for t in _on(s, Q.moe_route(xl, k, stream=s))]),
        "moe_swiglu": lambda s: Q.moe_swiglu(up, up, down, x, ids, p, stream=s),
    }

    def _on(s, outs):
        if s is not None:
            s.synchronize()
        return outs

    for name, call in calls.items():
        print(f"[case] busy current stream {name}", flush=True)
        want = call(None)
        side = _side()
        torch.cuda._sleep(BUSY)
        # blocks of the outputs' and the workspaces' sizes that the current
        # stream has let go of and is still to write to
        sizes = {want.numel() * want.element_size(), Q.gemm_workspace_size(w, xb), Q.moe_workspace_size(up, x, k), 4 * N * k}
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
        got = call(side)
        torch.cuda.synchronize()
        assert torch.equal(got, want), name


def test_gemm_noalloc_packed_tokens():
    print("[case] gemm_noalloc packed tokens", flush=True)
    for M, K, N in ((77, 96, 33), (300, 2048, 130)):
        w = Q.quantize(torch.randn((M, K), device=DEV), B.MXFP4)
        x = Q.quantize(torch.randn((N, K), device=DEV).bfloat16(), B.MXFP4)
        y = torch.full((N, M), 9.0, device=DEV)
        assert Q.gemm_noalloc(w, x, y) is y and torch.equal(y, Q.gemm(w, x))


def test_two_streams_in_a_graph():
    """Calls on a stream forked inside a capture, with outputs and workspaces of
    their own, beside calls on the capturing one: replays with new inputs equal
    the eager calls bit for bit."""
    print("[case] two streams in a graph", flush=True)
    K, M, N, E, k = 1024, 512, 6, 4, 2
    w = Q.quantize(torch.randn((M, 4 * K), device=DEV) * 0.05, B.Q4_0)
    up = Q.quantize_experts(torch.randn((E, M, K), device=DEV) * 0.05, B.MXFP4)
    down = Q.quantize_experts(torch.randn((E, K, M), device=DEV) * 0.05, B.MXFP4)
    x, xb = torch.empty((N, K), device=DEV), torch.empty((N, 4 * K), device=DEV, dtype=torch.bfloat16)
    logits = torch.empty((N, E), device=DEV)

    def calls(side):
        here = torch.cuda.current_stream()
        if side is not None:
            side.wait_stream(here)
        ids, p = Q.moe_route(logits, k, stream=side)
        outs = [ids, p, Q.moe_swiglu(up, up, down, x, ids, p, stream=side), Q.gemm(w, xb, stream=side), Q.gemv(w, xb.float()),
                Q.gemm(w, xb), Q.quantize(xb, B.MXFP4).data]
        if side is not None:
            here.wait_stream(side)
        return outs

    def fresh(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        for t in (x, xb, logits):
            t.copy_(torch.randn(t.shape, device=DEV, generator=g))

    fresh(0)
    assert Q.gemm_workspace_size(w, xb) > 0
    calls(None)
    capture, side = _side(), _side()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=capture):
        outs = calls(side)
    for seed in (1, 2, 3):
        fresh(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = calls(None)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"output {i}, seed {seed}"


def test_split_k_workspace_beside_a_busy_stream():
    """As test_calls_on_a_busy_streams_side, for a product that splits K."""
    print("[case] busy current stream, split K", flush=True)
    w, x = Q.quantize(torch.randn((256, 4096), device=DEV), B.Q4_0), torch.randn((200, 4096), device=DEV).bfloat16()
    n = Q.gemm_workspace_size(w, x)
    assert n > 0
    out, want = torch.empty((200, 256), device=DEV), Q.gemm(w, x)
    side = _side()
    torch.cuda._sleep(BUSY)
    torch.empty(n, dtype=torch.uint8, device=DEV).fill_(255)
    for _ in range(3):
        Q.gemm(w, x, out=out, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
