"""What the Python binding of the grouped products, the layer of many tokens and
the adapters refuses before anything is launched, and where it allocates, on
the CPU (the launch and the check for GPU tensors are replaced)."""
import pytest
import torch

import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B
from test_binding_checks import _Work, no_launch  # noqa: F401 (a fixture)

F32, F16, BF16, I32 = torch.float32, torch.float16, torch.bfloat16, torch.int32
E, K, F, M, N, k = 3, 64, 32, 48, 5, 2


def _experts(K, M, E=E, type_=B.MXFP4):
    return B.Experts(torch.zeros((E, M, B.row_size(type_, K)), dtype=torch.uint8), type_, K, M)


def _ops():
    return dict(w=_experts(K, M), x=torch.zeros((N, K), dtype=BF16), offsets=torch.zeros(E + 1, dtype=I32),
                order=torch.zeros(N * k, dtype=I32))


def test_group_refusals(no_launch):  # noqa: F811
    ids = torch.zeros((N, k), dtype=I32)
    for bad in (ids.long(), ids.float(), torch.zeros((k, N), dtype=I32).t(), torch.zeros((N, 2 * k), dtype=I32)[:, ::2]):
        with pytest.raises(ValueError, match="ids must be int32 and contiguous"):
            Q.moe_group(bad, E)
    for n in (0, -1, 1025):
        with pytest.raises(ValueError, match="n_experts"):
            Q.moe_group(ids, n)
    for ws in (torch.zeros((64, 4), dtype=torch.uint8)[:, 0], torch.zeros(1, dtype=torch.uint8).expand(64)):
        with pytest.raises(ValueError, match="workspace"):
            Q.moe_group(ids, E, workspace=ws)


@pytest.mark.parametrize("pair", [False, True])
def test_grouped_refusals(no_launch, pair):  # noqa: F811
    o = _ops()

    def call(w=o["w"], x=o["x"], offsets=o["offsets"], order=o["order"], **q):
        return Q.gemm_grouped_swiglu(w, w, x, offsets, order=order, top_k=k, **q) if pair else \
            Q.gemm_grouped(w, x, offsets, order=order, top_k=k, **q)

    for bad in (o["offsets"].long(), torch.zeros(2 * E + 2, dtype=I32)[::2]):
        with pytest.raises(ValueError, match="offsets must be int32"):
            call(offsets=bad)
    for n in (E, E + 2):
        with pytest.raises(ValueError, match="one value more"):
            call(offsets=torch.zeros(n, dtype=I32))
    for bad in (o["order"].long(), torch.zeros(4 * N, dtype=I32)[::2]):
        with pytest.raises(ValueError, match="order must be int32"):
            call(order=bad)
    with pytest.raises(ValueError, match="row of out"):
        call(out=torch.zeros((N * k + 1, M)))
    for t in (F16, torch.float64, torch.int32):
        with pytest.raises(ValueError, match="dtype must be"):
            call(dtype=t)
        with pytest.raises(ValueError, match="expected a torch.float32 tensor"):
            call(out=torch.zeros((N * k, M), dtype=t))
    for t in (F32, F16):
        with pytest.raises(ValueError, match="expected a torch.bfloat16 tensor"):
            call(x=o["x"].to(t))
    with pytest.raises(ValueError, match="contiguous"):
        call(x=torch.zeros((K, N), dtype=BF16).t())
    with pytest.raises(ValueError, match="packed weights"):
        call(w=B.Experts(o["w"].data, B.MXFP4, K, M + 1))


def test_layer_refusals(no_launch):  # noqa: F811
    g, d = _experts(K, F), _experts(F, M)
    x, ids, p = torch.zeros((N, K), dtype=BF16), torch.zeros((N, k), dtype=I32), torch.zeros((N, k))

    def call(x=x, ids=ids, p=p, **q):
        return Q.moe_gemm_swiglu(g, g, d, x, ids, p, **q)

    for q in (dict(ids=ids[:4]), dict(p=p[:4]), dict(ids=ids[0], p=p[0]), dict(p=p.double()), dict(p=torch.zeros((k, N)).t()),
              dict(x=x[:4])):
        with pytest.raises(ValueError, match=r"\(N, top_k\)"):
            call(**q)
    with pytest.raises(ValueError, match="ids must be int32"):
        call(ids=ids.long())
    with pytest.raises(ValueError, match="ids must be int32"):
        call(ids=torch.zeros((k, N), dtype=I32).t())
    with pytest.raises(ValueError, match="expected a torch.bfloat16 tensor"):
        call(x=x.float())
    with pytest.raises(ValueError, match="dtype must be"):
        call(dtype=F16)
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=torch.zeros((1 << 16, 2), dtype=torch.uint8)[:, 0])


def test_lora_refusals(no_launch):  # noqa: F811
    r, L = 16, 4
    a, b = torch.zeros((L, r, K), dtype=BF16), torch.zeros((L, M, r), dtype=BF16)
    x, ids = torch.zeros((N, K)), torch.zeros(N, dtype=I32)

    def call(a=a, b=b, x=x, ids=ids, **q):
        return Q.lora(a, b, x, ids, **q)

    for q in (dict(a=a.float()), dict(b=b.half()), dict(a=a[0]), dict(b=b[0])):
        with pytest.raises(ValueError, match="adapters must be bfloat16"):
            call(**q)
    for q in (dict(a=torch.zeros((L, K, r), dtype=BF16).transpose(1, 2)), dict(b=torch.zeros((L, M, 2 * r), dtype=BF16)[:, :, ::2])):
        with pytest.raises(ValueError, match="rows must be contiguous"):
            call(**q)
    for q in (dict(ids=ids[:4]), dict(ids=ids.view(N, 1)), dict(x=x[:4]), dict(x=x[0])):
        with pytest.raises(ValueError, match=r"ids must be \(N\)"):
            call(**q)
    with pytest.raises(ValueError, match="ids must be int32"):
        call(ids=ids.long())
    for t in (F16, torch.float64):
        with pytest.raises(ValueError, match="expected a torch.float32 tensor"):
            call(x=x.to(t))
    for s in (torch.zeros(L - 1), torch.zeros(L, dtype=F16), torch.zeros((L, 1)), torch.zeros(2 * L)[::2]):
        with pytest.raises(ValueError, match="scales must be"):
            call(scales=s)
    for t in (F16, BF16):
        with pytest.raises(ValueError, match="expected a torch.float32 tensor"):
            call(base=torch.zeros((N, M), dtype=t))
        with pytest.raises(ValueError, match="expected a torch.float32 tensor"):
            call(out=torch.zeros((N, M), dtype=t))
    with pytest.raises(ValueError, match="workspace"):
        call(workspace=torch.zeros((1 << 16, 2), dtype=torch.uint8)[:, 0])


def test_allocations_belong_to_the_stream(monkeypatch, qmm_lib):
    """Outputs and workspaces are allocated on the call's stream, and outputs are
    also kept for the caller's; without a stream nothing is switched or recorded."""
    o, g, d = _ops(), _experts(K, F), _experts(F, M)
    ids, p = torch.zeros((N, k), dtype=I32), torch.zeros((N, k))
    a, b = torch.zeros((4, 16, K), dtype=BF16), torch.zeros((4, M, 16), dtype=BF16)
    many, x, few = torch.zeros(66000, dtype=I32), torch.zeros((1100, K)), torch.zeros((2, K))
    calls = {
        "group": (3, lambda s: Q.moe_group(ids, E, stream=s)), "group of many": (4, lambda s: Q.moe_group(many, E, stream=s)),
        "grouped": (1, lambda s: Q.gemm_grouped(o["w"], o["x"], o["offsets"], stream=s)),
        "swiglu": (1, lambda s: Q.gemm_grouped_swiglu(g, g, o["x"], o["offsets"], order=o["order"], top_k=k, stream=s)),
        "layer": (2, lambda s: Q.moe_gemm_swiglu(g, g, d, o["x"], ids, p, stream=s)),
        "adapters": (2, lambda s: Q.lora(a, b, x, many[:1100], stream=s)),
        "adapters of few": (1, lambda s: Q.lora(a, b, few, many[:2], stream=s)),
    }
    for name, (made, call) in calls.items():
        with _Work(monkeypatch) as work:
            outs = call(work.stream)
        outs = list(outs) if isinstance(outs, (list, tuple)) else [outs]
        assert len(work.named("empty")) == made, name
        assert all(inside for _, inside in work.named("empty", "zeros", "zero_", "fill_")), name
        assert {(t.data_ptr(), "current") for t in outs} <= set(work.recorded), name
        assert [s for _, s in work.launched] == [work.stream], name
        with _Work(monkeypatch) as work:
            call(None)
        assert not any(inside for _, inside in work.ops) and not work.recorded, name


def test_shapes_of_what_is_made(monkeypatch, qmm_lib):
    """Strides that mean nothing (of empty tensors and single rows) are not refused."""
    launched = []
    monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
    monkeypatch.setattr(B, "_launch", lambda dev, stream, name, *args: launched.append(name))
    o = _ops()
    assert Q.gemm_grouped(o["w"], o["x"][:0], o["offsets"]).shape == (0, M)
    assert Q.gemm_grouped(o["w"], o["x"], o["offsets"], order=o["order"], top_k=k, dtype=BF16).dtype is BF16
    assert Q.gemm_grouped_swiglu(o["w"], o["w"], o["x"], o["offsets"]).dtype is BF16
    assert Q.gemm_grouped(o["w"], o["x"], o["offsets"], order=o["order"][:0]).shape == (0, M)
    a, b = torch.zeros((4, 16, 0), dtype=BF16), torch.zeros((4, 0, 16), dtype=BF16)
    assert Q.lora(a, b, torch.zeros((2, 0)), torch.zeros(2, dtype=I32)).shape == (2, 0)
    assert Q.lora(torch.zeros((1, 16, K), dtype=BF16), torch.zeros((1, M, 16), dtype=BF16), torch.zeros((0, K)),
                  torch.zeros(0, dtype=I32)).shape == (0, M)
    assert len(launched) == 6
