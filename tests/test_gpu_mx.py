"""The MXFP4 type on the GPU: quantization bit by bit, expansion, the decode
GEMV (alone, batched, fused with SwiGLU) and the prefill GEMM with bf16 and
with MXFP4 activations, against float64 references.

Every product is exact (an e2m1 value has two significant bits, its scale is a
power of two), so a sum of K terms may only be off by the binary32 accumulation:
at most (K + 64) 2^-24 sum |W' x| (the 64 covers the joining of partial sums),
and over many outputs the rounding errors, of random sign, leave a relative
2-norm error of about sqrt(3 K) 2^-24."""
import numpy as np
import pytest
import torch

import mx_ref as R
import quantized_matmul_ggml_amd as Q
from quantized_matmul_ggml_amd import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _weight(rows, K, pad=0):
    """Rows on the GPU, with `pad` more bytes per row that hold 0xFF."""
    if pad:
        rows = np.concatenate([rows, np.full((rows.shape[0], pad), 255, np.uint8)], 1)
    return B.Weight(torch.from_numpy(rows).to(DEV), B.MXFP4, K, rows.shape[0])


def _check(y, ref, a, K, what, norm=True):
    y = y.cpu().numpy().astype(np.float64)
    err, lim = np.abs(y - ref), (K + 64) * R.EPS * a + 1e-30
    bad = ~(err <= lim)
    assert not bad.any(), f"{what}: {bad.sum()} outputs off, worst {np.nanmax(err / lim)} of the bound"
    if norm and ref.size > 64:
        rel = np.linalg.norm(y - ref) / np.linalg.norm(ref)
        assert rel <= np.sqrt(3 * K) * R.EPS, f"{what}: relative error {rel}"


# ------------------------------------------------------------ quantization

def _adversarial(rng, M, K):
    """Blocks at many magnitudes: zeros, subnormals, exact ties, values at and
    next to powers of two, saturating values, signs of zero."""
    w = rng.standard_normal((M, K)).astype(np.float32) * np.exp2(rng.integers(-20, 20, (M, 1))).astype(np.float32)
    b = w.reshape(-1, 32)
    kind = rng.integers(0, 8, len(b))
    b[kind == 1] = 0.0
    b[kind == 2] *= np.float32(2.0 ** -120)
    b[kind == 3] = rng.choice(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.9999995], np.float32), (int((kind == 3).sum()), 32))
    t = b[kind == 3]
    t[:, 5] = 4.0
    b[kind == 3] = t * rng.choice(np.array([-1, 1], np.float32), t.shape)
    b[kind == 4] = np.float32(-0.0)
    t = b[kind == 5]
    t[:, 0] = np.nextafter(np.float32(8), np.float32(0))
    b[kind == 5] = t
    b[kind == 6] = b[kind == 6] * np.float32(2.0 ** -140)
    return w


@pytest.mark.parametrize("M,K,pad", [(1, 32, 0), (3, 64, 16), (37, 96, 0), (17, 544, 48), (64, 2048, 0), (5, 5632, 0)])
def test_quantize_bit_exact(M, K, pad):
    print(f"[case] mxfp4 quantize {M}x{K} pad {pad}", flush=True)
    w = _adversarial(np.random.default_rng(M + K), M, K)
    q = Q.quantize(torch.from_numpy(w).to(DEV), Q.MXFP4, pitch=Q.row_size(Q.MXFP4, K) + pad)
    rs = Q.row_size(Q.MXFP4, K)
    assert rs == R.row_size("mxfp4", K)
    rows = R.quantize_mxfp4(w)
    assert np.array_equal(q.data.cpu().numpy()[:, :rs], rows)
    back = Q.dequantize(q).cpu().numpy()
    want = R.values(rows, "mxfp4", K)
    assert np.array_equal(back.astype(np.float64), want)
    assert np.array_equal(np.signbit(back), np.signbit(want))
    # a value is off by at most half the widest step of its block (2 of amax's
    # 4 .. 8), and above 6 by up to 2
    amax = np.abs(w.reshape(-1, 32).astype(np.float64)).max(-1, keepdims=True)
    assert (np.abs(want - w).reshape(-1, 32) <= np.maximum(amax / 4, 2.0 ** -128)).all()


def test_quantize_bf16_rows():
    print("[case] mxfp4 quantize bf16", flush=True)
    rng = np.random.default_rng(5)
    for M, K, stride in ((1, 32, 32), (77, 2048, 2048), (9, 160, 192)):
        x = torch.from_numpy(_adversarial(rng, M, stride)).to(torch.bfloat16).to(DEV)[:, :K]
        rows = R.quantize_mxfp4(x.float().cpu().numpy())
        assert np.array_equal(Q.quantize(x, Q.MXFP4).data.cpu().numpy(), rows)


def test_blocks_that_are_not_finite():
    """A block with an infinity or a NaN has scale byte 255 and no codes; it
    expands to NaN and gives NaN in every product it meets, and nowhere else."""
    print("[case] mxfp4 not finite", flush=True)
    w = np.random.default_rng(1).standard_normal((40, 96)).astype(np.float32)
    w[3, 40], w[7, 2], w[9, 95] = np.inf, np.nan, -np.inf
    q = Q.quantize(torch.from_numpy(w).to(DEV), Q.MXFP4)
    rows = R.quantize_mxfp4(w)
    assert np.array_equal(q.data.cpu().numpy(), rows)
    want = R.values(rows, "mxfp4", 96)
    back = Q.dequantize(q).cpu().numpy()
    assert np.array_equal(np.isnan(back), np.isnan(want)) and np.isnan(want).sum() == 96
    bad = np.isin(np.arange(40), (3, 7, 9))
    x = torch.ones((20, 96), device=DEV)
    for y in (Q.gemv(q, x[:8]), Q.gemv(q, x[:1]), Q.gemm(q, x.bfloat16()), Q.gemm(q, Q.quantize(x, Q.MXFP4))):
        assert np.array_equal(np.isnan(y.cpu().numpy()), np.broadcast_to(bad, y.shape))


# ------------------------------------------------------------- decode GEMV

GEMV = [(1, 32), (15, 64), (16, 96), (17, 128), (33, 160), (256, 544), (100, 2048), (2047, 2080), (4100, 512),
        (48, 5632), (70, 11008), (20, 32768), (9000, 256)]


@pytest.mark.parametrize("M,K", GEMV)
def test_gemv(M, K):
    rng = np.random.default_rng(1000 * M + K)
    rows = R.random_rows(rng, "mxfp4", (M,), K)
    w, W = _weight(rows, K, pad=32 * (M % 2)), R.values(rows, "mxfp4", K)
    for N in (1, 2, 3, 4, 5, 8) if M * K < 1 << 22 else (1, 4, 7):
        print(f"[case] mxfp4 gemv {M}x{K} N {N}", flush=True)
        x = (rng.standard_normal((N, K)) * np.exp2(rng.integers(-9, 9, (N, K))) + 1.0).astype(np.float32)
        y = Q.gemv(w, torch.from_numpy(x).to(DEV))
        x = x.astype(np.float64)
        _check(y, x @ W.T, np.abs(x) @ np.abs(W).T, K, f"N {N}", norm=False)


@pytest.mark.parametrize("M,K,N", [(70001, 160, 1), (70001, 160, 8), (70001, 1056, 3), (33000, 5664, 2), (33000, 2080, 7)])
def test_gemv_more_tiles_than_workgroups(M, K, N):
    """Workgroups take several tiles each, with one and with several passes over
    K; rows at both ends and in between against the reference."""
    print(f"[case] mxfp4 gemv {M}x{K} N {N}", flush=True)
    rng = np.random.default_rng(M + K + N)
    some = R.random_rows(rng, "mxfp4", (97,), K)
    at = np.unique(np.concatenate([np.arange(40), np.arange(M - 40, M), rng.integers(0, M, 400)]))
    rows = some[np.arange(M) % 97]
    w, W = _weight(rows, K), R.values(some, "mxfp4", K)[at % 97]
    x = rng.standard_normal((N, K)).astype(np.float32)
    y = Q.gemv(w, torch.from_numpy(x).to(DEV))
    x = x.astype(np.float64)
    _check(y[:, torch.from_numpy(at).to(DEV)], x @ W.T, np.abs(x) @ np.abs(W).T, K, "some rows", norm=False)
    # the rows repeat, and so do the results, bit for bit
    assert torch.equal(y[:, :M - 97], y[:, 97:])


def test_gemv_relative_error():
    """Gaussian activations: the relative error of the whole product."""
    print("[case] mxfp4 gemv relative error", flush=True)
    rng = np.random.default_rng(3)
    for M, K, N in ((512, 2048, 1), (300, 5632, 8)):
        rows = R.random_rows(rng, "mxfp4", (M,), K)
        W, x = R.values(rows, "mxfp4", K), rng.standard_normal((N, K)).astype(np.float32)
        y = Q.gemv(_weight(rows, K), torch.from_numpy(x).to(DEV))
        x = x.astype(np.float64)
        _check(y, x @ W.T, np.abs(x) @ np.abs(W).T, K, f"{M}x{K}")


def test_gemv_strides_and_untouched_bytes():
    """Token rows inside a wider buffer at a 4-byte aligned address, outputs
    with a pitch: the bytes between the outputs stay as they were."""
    print("[case] mxfp4 gemv strides", flush=True)
    rng = np.random.default_rng(8)
    M, K, N = 77, 608, 6
    rows = R.random_rows(rng, "mxfp4", (M,), K)
    big = torch.randn((N, K + 9), device=DEV)
    x = big[:, 3:3 + K]
    out = torch.full((N, M + 5), 7.0, device=DEV)
    Q.gemv(_weight(rows, K), x, out=out[:, 2:2 + M])
    W, xd = R.values(rows, "mxfp4", K), x.double().cpu().numpy()
    _check(out[:, 2:2 + M], xd @ W.T, np.abs(xd) @ np.abs(W).T, K, "strides", norm=False)
    o = out.cpu().numpy()
    assert (o[:, :2] == 7).all() and (o[:, 2 + M:] == 7).all()


def test_gemv_special_activations():
    """Zeros give zeros; an infinite or NaN activation stays in its own token."""
    print("[case] mxfp4 gemv special activations", flush=True)
    rng = np.random.default_rng(9)
    M, K = 50, 320
    rows = R.random_rows(rng, "mxfp4", (M,), K)
    W = R.values(rows, "mxfp4", K)
    x = rng.standard_normal((5, K)).astype(np.float32)
    x[0], x[2, 7], x[3, 11] = 0, np.inf, np.nan
    x[4] *= np.float32(1e38)
    y = Q.gemv(_weight(rows, K), torch.from_numpy(x).to(DEV)).cpu().numpy()
    assert (y[0] == 0).all() and np.isnan(y[3]).all()
    nz = W[:, 7] != 0
    assert np.array_equal(y[2][nz], np.where(W[nz, 7] > 0, np.inf, -np.inf)) and np.isnan(y[2][~nz]).all()
    # A binary32 sum stays finite in every order only if its magnitudes add up
    # to less than 2^128 (a partial sum is at most that large, and one above is
    # an infinity): token 4's rows above that may be infinite, the others not.
    for n in (1, 4):
        xd = x[n].astype(np.float64)
        a = np.abs(W) @ np.abs(xd)
        good = np.abs(y[n] - W @ xd) <= (K + 64) * R.EPS * a + 1e-30
        assert (good | ((a >= 2.0 ** 128) & ~np.isfinite(y[n]))).all()
    # large activations whose sums stay far below it
    big = x[1] * np.float32(1e35)
    y, xd = Q.gemv(_weight(rows, K), torch.from_numpy(big[None]).to(DEV)).cpu().numpy()[0], big.astype(np.float64)
    a = np.abs(W) @ np.abs(xd)
    assert a.max() < 2.0 ** 126 and (np.abs(y - W @ xd) <= (K + 64) * R.EPS * a).all()


def test_gemv_k_zero():
    print("[case] mxfp4 gemv K 0", flush=True)
    w = B.Weight(torch.empty((5, 16), dtype=torch.uint8, device=DEV), B.MXFP4, 0, 5)      # rows 16 bytes apart
    y = torch.full((2, 5), 3.0, device=DEV)
    Q.gemv(w, torch.empty((2, 0), device=DEV), out=y)
    assert (y == 0).all()


def test_gemv_batch_and_swiglu():
    rng = np.random.default_rng(10)
    for K, Ms, N in ((256, (40, 1, 130), 1), (2048, (300, 64), 8), (4128, (17, 2000, 16), 3)):
        print(f"[case] mxfp4 gemv batch K {K} N {N}", flush=True)
        rows = [R.random_rows(rng, "mxfp4", (M,), K) for M in Ms]
        xs = [rng.standard_normal((N, K)).astype(np.float32) for _ in Ms]
        ys = Q.gemv_batch([(_weight(r, K), torch.from_numpy(x).to(DEV), None) for r, x in zip(rows, xs)])
        for r, x, y in zip(rows, xs, ys):
            W, xd = R.values(r, "mxfp4", K), x.astype(np.float64)
            _check(y, xd @ W.T, np.abs(xd) @ np.abs(W).T, K, f"batch K {K}", norm=False)
    for M, K, N in ((1, 32, 1), (9, 96, 2), (1000, 2048, 1), (301, 2048, 8), (24, 8192, 5)):
        print(f"[case] mxfp4 gemv swiglu {M}x{K} N {N}", flush=True)
        g, u = R.random_rows(rng, "mxfp4", (M,), K), R.random_rows(rng, "mxfp4", (M,), K)
        x = (rng.standard_normal((N, K)) * 0.1).astype(np.float32)
        h = Q.gemv_swiglu(_weight(g, K), _weight(u, K, pad=16), torch.from_numpy(x).to(DEV)).cpu().numpy()
        G, U, xd = R.values(g, "mxfp4", K), R.values(u, "mxfp4", K), x.astype(np.float64)
        gs, us = xd @ G.T, xd @ U.T
        eg = (K + 64) * R.EPS * (np.abs(xd) @ np.abs(G).T)
        eu = (K + 64) * R.EPS * (np.abs(xd) @ np.abs(U).T)
        ref = R.swish(gs) * us
        lim = 1.1 * eg * (np.abs(us) + eu) + np.abs(R.swish(gs)) * eu + 2.0 ** -20 * np.abs(ref) + 1e-30
        assert (np.abs(h - ref) <= lim).all()


# ------------------------------------------------------------ prefill GEMM

GEMM = [(1, 32, 1), (5, 96, 9), (33, 64, 70), (128, 256, 128), (129, 288, 127), (300, 2048, 77), (257, 1056, 300),
        (100, 5632, 40), (700, 512, 513)]


@pytest.mark.parametrize("M,K,N", GEMM)
def test_gemm_bf16(M, K, N):
    print(f"[case] mxfp4 gemm bf16 {M}x{K}x{N}", flush=True)
    rng = np.random.default_rng(M + K + N)
    rows = R.random_rows(rng, "mxfp4", (M,), K)
    x = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).to(torch.bfloat16)
    w, W, xd = _weight(rows, K, pad=16), R.values(rows, "mxfp4", K), x.double().numpy()
    ref, a = xd @ W.T, np.abs(xd) @ np.abs(W).T
    for ws in ("auto", None):
        _check(Q.gemm(w, x.to(DEV), workspace=ws), ref, a, K, f"workspace {ws}")
    out = torch.empty((N, M), device=DEV)
    _check(Q.gemm_noalloc(w, x.to(DEV), out), ref, a, K, "noalloc")


def test_gemm_bf16_batch_and_swiglu():
    rng = np.random.default_rng(20)
    K, N = 1120, 90
    print("[case] mxfp4 gemm batch", flush=True)
    rows = [R.random_rows(rng, "mxfp4", (M,), K) for M in (130, 40)]
    x = torch.from_numpy((0.1 * rng.standard_normal((N, K))).astype(np.float32)).to(torch.bfloat16)
    ws = [_weight(r, K) for r in rows]
    xg = x.to(DEV)
    ys = Q.gemm_batch([(w, xg, None) for w in ws])
    for w, y in zip(ws, ys):
        assert torch.equal(y, Q.gemm(w, xg, workspace=None))
    print("[case] mxfp4 gemm swiglu", flush=True)
    g, u = (R.random_rows(rng, "mxfp4", (100,), K) for _ in range(2))
    h = Q.gemm_swiglu(_weight(g, K), _weight(u, K), xg).cpu().numpy()
    G, U, xd = R.values(g, "mxfp4", K), R.values(u, "mxfp4", K), x.double().numpy()
    gs, us = xd @ G.T, xd @ U.T
    eg, eu = (K + 64) * R.EPS * (np.abs(xd) @ np.abs(G).T), (K + 64) * R.EPS * (np.abs(xd) @ np.abs(U).T)
    ref = R.swish(gs) * us
    assert (np.abs(h - ref) <= 1.1 * eg * (np.abs(us) + eu) + np.abs(R.swish(gs)) * eu + 2.0 ** -20 * np.abs(ref) + 1e-30).all()


@pytest.mark.parametrize("M,K,N", GEMM + [(4100, 544, 4099)])
def test_gemm_mx(M, K, N):
    print(f"[case] mxfp4 gemm mx {M}x{K}x{N}", flush=True)
    rng = np.random.default_rng(M * K + N)
    rows, xr = R.random_rows(rng, "mxfp4", (M,), K), R.random_rows(rng, "mxfp4", (N,), K)
    w, x = _weight(rows, K, pad=16), _weight(xr, K, pad=48)
    W, X = R.values(rows, "mxfp4", K), R.values(xr, "mxfp4", K)
    ref, a = X @ W.T, np.abs(X) @ np.abs(W).T
    out = torch.full((N, M + 3), 5.0, device=DEV)
    Q.gemm(w, x, out=out[:, 1:1 + M])
    _check(out[:, 1:1 + M], ref, a, K, "mx")
    o = out.cpu().numpy()
    assert (o[:, 0] == 5).all() and (o[:, 1 + M:] == 5).all()
    if N < 600:
        ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)       # accepted, not used
        _check(Q.gemm(w, x, workspace=ws), ref, a, K, "mx with a workspace")
        y = torch.empty((N, M), device=DEV)
        B._check(B.lib().qmm_gemm_noalloc(*(B.ctypes.byref(d) for d in (w.desc(), x.desc(), B._dense_desc(y, B.F32))),
                                          0, B._stream(None)), "qmm_gemm_noalloc")
        _check(y, ref, a, K, "mx noalloc")


@pytest.mark.parametrize("M,K,N", [(1700, 544, 1500), (1701, 96, 1499), (1650, 2080, 1590), (1537, 32, 1537)])
def test_gemm_mx_middle_sizes(M, K, N):
    """Enough tiles of 64 x 64 for tiles of 128 x 128, too few for 256 x 256."""
    test_gemm_mx(M, K, N)


def test_gemm_mx_extreme_scales():
    """Scales at both ends of the range: products of 2^-127 and 2^127."""
    print("[case] mxfp4 gemm mx extreme scales", flush=True)
    rng = np.random.default_rng(4)
    M, K, N = 40, 64, 36
    rows, xr = R.random_rows(rng, "mxfp4", (M,), K), R.random_rows(rng, "mxfp4", (N,), K)
    rows[:, :2], xr[:, :2] = [[0, 10]], [[254, 244]]
    W, X = R.values(rows, "mxfp4", K), R.values(xr, "mxfp4", K)
    _check(Q.gemm(_weight(rows, K), _weight(xr, K)), X @ W.T, np.abs(X) @ np.abs(W).T, K, "extreme")
    x = np.exp2(rng.integers(100, 120, (4, K))).astype(np.float32)
    rows[:, :2] = [[0, 3]]
    W = R.values(rows, "mxfp4", K)
    _check(Q.gemv(_weight(rows, K), torch.from_numpy(x).to(DEV)), x.astype(np.float64) @ W.T,
           x.astype(np.float64) @ np.abs(W).T, K, "extreme gemv", norm=False)


def test_streams_and_graph():
    """On another stream, and captured into a graph: replays with new inputs
    equal the eager calls bit for bit."""
    print("[case] mxfp4 graph", flush=True)
    M, K = 600, 2048
    w = Q.quantize(torch.randn((M, K), device=DEV) * 0.02, Q.MXFP4)
    x, xb = torch.empty((5, K), device=DEV), torch.empty((200, K), device=DEV, dtype=torch.bfloat16)
    names = ("gemv", "swiglu", "gemm", "mx", "deq")

    def calls():
        xq = Q.quantize(xb, Q.MXFP4)
        return dict(zip(names, (Q.gemv(w, x), Q.gemv_swiglu(w, w, x), Q.gemm(w, xb), Q.gemm(w, xq), Q.dequantize(xq))))

    def fresh(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(x.shape, device=DEV, generator=g))
        xb.copy_(torch.randn(xb.shape, device=DEV, generator=g))

    fresh(1)
    ref = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = calls()
    side.synchronize()
    for n in names:
        assert torch.equal(ref[n], other[n]), n
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = calls()
    for seed in (2, 3, 4):
        fresh(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = calls()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(ref[n], outs[n]), f"{n}, seed {seed}"
