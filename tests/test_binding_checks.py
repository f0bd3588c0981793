"""What the Python binding refuses before anything is launched, on the CPU:
the launch itself and the check for GPU tensors are replaced, so that a call
which gets past the binding's own checks fails the test."""
import contextlib
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B


@pytest.fixture
def no_launch(monkeypatch, qmm_lib):
    def launch(dev, stream, name, *args):
        pytest.fail(f"{name} was launched")

    monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
    monkeypatch.setattr(B, "_launch", launch)


def _weight(type_=B.MXFP4, K=64, M=32):
    return B.Weight(torch.zeros((M, B.row_size(type_, K)), dtype=torch.uint8), type_, K, M)


# ----------------------------------------------------------- element types

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.mark.parametrize("N", [1, 4])
def test_element_types(no_launch, N):
    """Operands of another element type, of one row too (whose pitch the
    library does not look at)."""
    w, K, M = _weight(), 64, 32
    x = {t: torch.zeros((N, K), dtype=t) for t in (F32, F16, BF16, torch.float64)}
    y = {t: torch.zeros((N, M), dtype=t) for t in (F32, F16, BF16)}
    calls = []
    for t in (F16, BF16, torch.float64):
        calls += [lambda t=t: Q.gemv(w, x[t]), lambda t=t: Q.gemv_swiglu(w, w, x[t]), lambda t=t: Q.gemv_batch([(w, x[t], None)])]
    for t in (F32, F16):
        calls += [lambda t=t: Q.gemm(w, x[t]), lambda t=t: Q.gemm(w, x[t], workspace=None), lambda t=t: Q.gemm_swiglu(w, w, x[t]),
                  lambda t=t: Q.gemm_batch([(w, x[t], None)]), lambda t=t: Q.gemm_noalloc(w, x[t], y[F32]),
                  lambda t=t: Q.gemm_workspace_size(w, x[t])]
    for t in (F16, BF16):
        calls += [lambda t=t: Q.gemv(w, x[F32], out=y[t]), lambda t=t: Q.gemv_swiglu(w, w, x[F32], out=y[t]),
                  lambda t=t: Q.gemv_batch([(w, x[F32], y[t])]), lambda t=t: Q.gemm(w, x[BF16], out=y[t]),
                  lambda t=t: Q.gemm(w, x[BF16], out=y[t], workspace=None), lambda t=t: Q.gemm_swiglu(w, w, x[BF16], out=y[t]),
                  lambda t=t: Q.gemm_batch([(w, x[BF16], y[t])]), lambda t=t: Q.gemm_noalloc(w, x[BF16], y[t]),
                  lambda t=t: Q.gemv(w, _weight(B.Q8_0, K, N), out=y[t]),
                  lambda t=t: Q.dequantize(_weight(M=N), out=torch.zeros((N, K), dtype=t))]
    for call in calls:
        with pytest.raises(ValueError, match="expected a torch.(float32|bfloat16) tensor"):
            call()


# ---------------------------------------------------- sizes the caller gives

def test_pitch_below_the_row(no_launch):
    for type_ in (B.MXFP4, B.Q4_0, B.Q8_0):
        rs = Q.row_size(type_, 64)
        for M in (1, 3):
            with pytest.raises(ValueError, match="below the row"):
                Q.quantize(torch.zeros((M, 64)), type_, pitch=rs - 16)
            if type_ != B.MXFP4:
                with pytest.raises(ValueError, match="below the row"):
                    Q.records_to_rows(torch.zeros(1 << 12, dtype=torch.uint8), type_, 64, M, pitch=rs - 16)


def test_buffers_too_small_or_with_holes(no_launch):
    w = _weight(B.Q4_0)
    n = 32 * 2 * 18
    byte = lambda k: torch.zeros(k, dtype=torch.uint8)
    wide = byte(4 * n).view(n, 4)[:, 0]                 # n bytes, four apart
    one = byte(1).expand(n)
    for bad in (byte(n - 1), wide, one):
        with pytest.raises(ValueError, match="records"):
            Q.records_to_rows(bad, B.Q4_0, 64, 32)
        with pytest.raises(ValueError, match="out"):
            Q.rows_to_records(w, out=bad)
    sink = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="src"):
        Q.stream_read(byte(64), sink, nbytes=80, workgroups=8)
    with pytest.raises(ValueError, match="src"):
        Q.stream_read(wide, sink, workgroups=8)
    with pytest.raises(ValueError, match="sink"):
        Q.stream_read(byte(64), sink, workgroups=9)
    x = torch.zeros((4, 64), dtype=BF16)
    for ws in (wide, one):
        with pytest.raises(ValueError, match="workspace"):
            Q.gemm(w, x, workspace=ws)
        ex = Q.Experts(torch.zeros((2, 64, Q.row_size(B.Q4_0, 64)), dtype=torch.uint8), B.Q4_0, 64, 64)
        with pytest.raises(ValueError, match="workspace"):
            Q.moe_swiglu(ex, ex, ex, x.float(), torch.zeros((4, 1), dtype=torch.int32), torch.zeros((4, 1)), workspace=ws)


def test_weights_that_their_data_does_not_hold(no_launch):
    """More rows than the data has (a row range past the end among them), a
    single row or rows of a view that are shorter than K weights, and elements that are apart."""
    K, x = 64, torch.zeros((1, 64))
    rs = Q.row_size(B.MXFP4, K)
    data = torch.zeros((32, rs), dtype=torch.uint8)
    apart = torch.zeros((32, 2 * rs), dtype=torch.uint8)[:, ::2]
    for w in (B.Weight(data, B.MXFP4, K, 33), B.Weight(data, B.MXFP4, K, 32).rows(8, 40), B.Weight(data[:1, :16], B.MXFP4, K, 1),
              B.Weight(data[:, :rs - 16], B.MXFP4, K, 32), B.Weight(apart, B.MXFP4, K, 32), B.Weight(apart.t(), B.MXFP4, K, 32),
              B.Weight(torch.zeros((1, K - 1), dtype=torch.float16), B.F16, K, 1)):
        for call in (lambda: Q.gemv(w, x), lambda: Q.gemm(w, x.bfloat16()), lambda: Q.gemv_batch([(w, x, None)]), w.desc,
                     lambda: Q.dequantize(w), lambda: Q.rows_to_records(w)):
            with pytest.raises(ValueError, match="packed weights"):
                call()
    good = B.Experts(torch.zeros((2, K, rs), dtype=torch.uint8), B.MXFP4, K, K)
    ids, p = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 1))
    for bad in (B.Experts(data.view(2, 16, rs), B.MXFP4, K, 17), B.Experts(data[:, :16].unsqueeze(1), B.MXFP4, K, 1),
                B.Experts(data.view(2, 16, rs)[:, :, :16], B.MXFP4, K, 16), B.Experts(apart.unsqueeze(0), B.MXFP4, K, 32)):
        for args in ((bad, good, good), (good, bad, good), (good, good, bad)):
            with pytest.raises(ValueError, match="packed weights"):
                Q.moe_swiglu(*args, x, ids, p)
        with pytest.raises(ValueError, match="packed weights"):
            bad.desc()
    assert bytes(good.desc()) == good._desc()


# ------------------------------------------------------------------ streams

class _Work(TorchDispatchMode):
    """The torch operators that run inside and outside the fake stream."""

    def __init__(self, monkeypatch):
        super().__init__()
        self.stream = types.SimpleNamespace(cuda_stream=7, device_index=0)
        self.inside, self.ops, self.launched, self.recorded = False, [], [], []

        @contextlib.contextmanager
        def on(stream):
            assert stream is self.stream
            self.inside = True
            yield
            self.inside = False

        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: "current")
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: self.recorded.append((t.data_ptr(), s)))
        monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
        monkeypatch.setattr(B, "_launch", lambda dev, stream, name, *args: self.launched.append((name, stream)))

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.ops.append((func.overloadpacket.__name__, self.inside))
        return func(*args, **(kwargs or {}))

    def named(self, *names):
        return [o for o in self.ops if o[0] in names]


@pytest.mark.parametrize("layout", ["rows", "transposed", "gaps"])
def test_quantize_experts_copies_on_its_stream(monkeypatch, qmm_lib, layout):
    """Matrices whose rows cannot be one list are copied, on the call's stream:
    on another one the quantizer could read the copy before it is made."""
    w = {"rows": torch.randn(3, 8, 64), "transposed": torch.randn(3, 64, 8).transpose(1, 2), "gaps": torch.randn(3, 9, 64)[:, :8]}[layout]
    with _Work(monkeypatch) as work:
        q = Q.quantize_experts(w, B.MXFP4, stream=work.stream)
    assert (q.K, q.M, q.data.shape) == (64, 8, (3, 8, Q.row_size(B.MXFP4, 64)))
    copies = work.named("clone", "copy_", "_to_copy")
    assert len(copies) == (0 if layout == "rows" else 1) and all(inside for _, inside in copies)
    assert work.launched == [("qmm_quantize_rule", work.stream)]


def test_allocations_belong_to_the_stream(monkeypatch, qmm_lib):
    """Outputs and workspaces are allocated (and cleared) on the call's stream,
    and outputs are also kept for the caller's; without a stream nothing is
    switched or recorded."""
    K, M, N = 4096, 64, 5
    w, q4 = _weight(K=K, M=M), _weight(B.Q4_0, K, M)
    x, xb, rs = torch.zeros((N, K)), torch.zeros((N, K), dtype=BF16), Q.row_size(B.Q4_0, K)
    ex = B.Experts(torch.zeros((2, 64, Q.row_size(B.MXFP4, 64)), dtype=torch.uint8), B.MXFP4, 64, 64)
    ids, p, x64 = torch.zeros((N, 1), dtype=torch.int32), torch.zeros((N, 1)), torch.zeros((N, 64))
    w3 = torch.zeros((2, 3, 64))
    rec = torch.zeros(M * K // 32 * 18, dtype=torch.uint8)
    assert Q.gemm_workspace_size(q4, xb) > 0
    calls = {
        "quantize": (1, lambda s: Q.quantize(x, B.Q4_0, pitch=rs + 16, stream=s).data),
        "quantize_experts": (1, lambda s: Q.quantize_experts(w3, B.MXFP4, stream=s).data),
        "dequantize": (1, lambda s: Q.dequantize(w, stream=s)),
        "gemv": (1, lambda s: Q.gemv(w, x, stream=s)),
        "gemv_batch": (2, lambda s: Q.gemv_batch([(w, x, None), (w, x, None)], stream=s)),
        "gemv_swiglu": (1, lambda s: Q.gemv_swiglu(w, w, x, stream=s)),
        "records_to_rows": (1, lambda s: Q.records_to_rows(rec, B.Q4_0, K, M, stream=s).data),
        "rows_to_records": (1, lambda s: Q.rows_to_records(q4, stream=s)),
        "gemm": (2, lambda s: Q.gemm(q4, xb, stream=s)),                     # its split-K workspace too
        "gemm_swiglu": (1, lambda s: Q.gemm_swiglu(w, w, xb, stream=s)),
        "gemm_batch": (2, lambda s: Q.gemm_batch([(w, xb, None), (w, xb, None)], stream=s)),
        "moe_route": (2, lambda s: Q.moe_route(x64, 1, stream=s)),
        "moe_swiglu": (2, lambda s: Q.moe_swiglu(ex, ex, ex, x64, ids, p, stream=s)),
    }
    for name, (made, call) in calls.items():
        with _Work(monkeypatch) as work:
            outs = call(work.stream)
        outs = list(outs) if isinstance(outs, (list, tuple)) else [outs]
        assert len(work.named("empty")) == made, name
        assert all(inside for _, inside in work.named("empty", "zeros", "zero_", "fill_")), name
        assert {(o.data_ptr(), "current") for o in outs} <= set(work.recorded), name
        assert [s for _, s in work.launched] == [work.stream], name
        with _Work(monkeypatch) as work:
            call(None)
        assert not any(inside for _, inside in work.ops) and not work.recorded, name


def test_stream_of_another_gpu(monkeypatch, qmm_lib):
    """A stream of another GPU than the tensors' is refused, also by the
    measuring read (which launched on the current GPU, whatever its tensors')."""
    other = types.SimpleNamespace(cuda_stream=7, device_index=1)
    with pytest.raises(ValueError, match="stream of GPU 1"):
        B._launch(0, other, "qmm_gemv", None, None, None)
    monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
    with pytest.raises(ValueError, match="stream of GPU 1"):
        Q.stream_read(torch.zeros(64, dtype=torch.uint8), torch.zeros(8, dtype=torch.int32), workgroups=8, stream=other)


def test_packed_tokens_of_every_gemm_form(monkeypatch, qmm_lib):
    """gemm_noalloc and gemm_workspace_size take packed tokens, as gemm does."""
    w, x, y = _weight(), _weight(M=5), torch.zeros((5, 32))
    launched = []
    monkeypatch.setattr(B, "_need_gpu", lambda *ts: 0)
    monkeypatch.setattr(B, "_launch", lambda dev, stream, name, *args: launched.append((name, *args)))
    assert Q.gemm_workspace_size(w, x) == 0
    assert Q.gemm_noalloc(w, x, y) is y
    assert launched == [("qmm_gemm_noalloc", w._desc(), x._desc(), B._dense(y, B.F32), 0)]


def test_weights_of_no_rows(qmm_lib):
    """Strides of empty data mean nothing (torch gives (1, M) to a transposed
    one, and arrays from elsewhere bring zeros)."""
    for data, type_ in ((torch.zeros((0, 64), dtype=torch.float16).as_strided((0, 64), (0, 0)), B.F16),
                        (torch.zeros((64, 0), dtype=torch.uint8).t(), B.MXFP4)):
        d = B.Weight(data, type_, 64, 0).desc()
        assert (d.ne[0], d.ne[1]) == (64, 0)
    d = B.Experts(torch.zeros((48, 0, 3), dtype=torch.uint8).permute(2, 1, 0), B.MXFP4, 64, 0).desc()
    assert (d.ne[0], d.ne[1], d.ne[2]) == (64, 0, 3)
