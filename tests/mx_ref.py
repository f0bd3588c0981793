"""Plain float64 / bit-level references for the MXFP4 type and the
mixture-of-experts layer (numpy on the CPU, written from the formats and
formulas in include/qmm.h; no code shared with the library)."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([E2M1, -E2M1])
EPS = 2.0 ** -24        # half a step of binary32, relative


def align16(n):
    return (n + 15) // 16 * 16


def row_size(kind, K):
    if kind == "mxfp4":
        return align16(K // 32) + K // 2
    if kind in ("q4_0", "q8_0"):
        return align16(K // 16) + (K // 2 if kind == "q4_0" else K)
    return align16(K // 32) + (K // 2 if kind == "q4_b64" else K)


def nearest_code(a):
    """e2m1 code (0..7) nearest to the magnitude a, one value at a time: the
    smaller distance, on a tie the even code, above the largest value 7."""
    d = np.abs(E2M1 - a)
    best = int(np.argmin(d))
    if best < 7 and d[best + 1] == d[best]:
        best += best & 1
    return best


def quantize_mxfp4(w):
    """float32 (M, K) -> MXFP4 rows, block by block."""
    M, K = w.shape
    out = np.zeros((M, row_size("mxfp4", K)), np.uint8)
    qoff = align16(K // 32)
    for r in range(M):
        for b in range(K // 32):
            v = w[r, 32 * b:32 * b + 32].astype(np.float64)
            if not np.isfinite(v).all():
                out[r, b] = 255
                continue
            amax = np.abs(v).max()
            e = -127 if amax == 0 else max(int(np.frexp(amax)[1]) - 3, -127)
            out[r, b] = e + 127
            c = [nearest_code(x) | (8 if s else 0) for x, s in zip(np.abs(v) * 2.0 ** -e, np.signbit(v))]
            out[r, qoff + 16 * b:qoff + 16 * b + 16] = [c[j] | c[j + 16] << 4 for j in range(16)]
    return out


def values(rows, kind, K):
    """Packed rows (..., bytes) -> float64 (..., K)."""
    n = K // (64 if kind.endswith("b64") else 32)
    if kind == "mxfp4":
        s = rows[..., :n].astype(np.float64)
        d = np.where(s == 255, np.nan, np.exp2(s - 127))
        off = align16(n)
    else:
        d = np.ascontiguousarray(rows[..., :2 * n]).view(np.float16).astype(np.float64)
        off = align16(2 * n)
    if kind in ("q8_0", "q8_b64"):
        q = np.ascontiguousarray(rows[..., off:off + K]).view(np.int8).astype(np.float64)
    else:
        by = rows[..., off:off + K // 2].reshape(*rows.shape[:-1], K // 32, 16)
        c = np.concatenate([by & 15, by >> 4], -1)
        q = VALUES[c] if kind == "mxfp4" else c.astype(np.float64) - 8
        q = q.reshape(*rows.shape[:-1], K)
    return q * np.repeat(d, K // n, -1)


def random_rows(rng, kind, shape, K, spread=4):
    """Random packed rows (shape..., bytes), every code possible, scales over
    2 * spread binades around those of trained weights; padding bytes set."""
    rs = row_size(kind, K)
    rows = rng.integers(0, 256, (*shape, rs), dtype=np.uint8)
    n = K // (64 if kind.endswith("b64") else 32)
    if kind == "mxfp4":
        rows[..., :n] = rng.integers(120 - spread, 120 + spread, (*shape, n))
    else:
        s = (np.exp2(rng.uniform(-7 - spread / 2, -7 + spread / 2, (*shape, n)))).astype(np.float16)
        rows[..., :2 * n] = s.view(np.uint8)
        if kind.startswith("q8"):           # codes -127 .. 127
            off = align16(2 * n)
            c = rows[..., off:off + K]
            c[c == 128] = 129
    return rows


def swish(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def route(logits, k, rule_all):
    """(ids, weights) of qmm_moe_route, token by token."""
    N, E = logits.shape
    ids, w = np.full((N, k), -1, np.int32), np.zeros((N, k))
    for n in range(N):
        l = [(float(v), e) for e, v in enumerate(logits[n]) if v > -np.inf]
        if not l:
            continue
        top = max(v for v, _ in l)
        p = {e: 1.0 if v == top else float(np.exp(v - top)) for v, e in l}
        order = sorted(l, key=lambda t: (-t[0], t[1]))[:k]
        total = sum(p.values()) if rule_all else sum(p[e] for _, e in order)
        for s, (_, e) in enumerate(order):
            ids[n, s], w[n, s] = e, p[e] / total
    return ids, w


def moe(gate, up, down, x, ids, weights):
    """(y, bound): float64 layer over dequantized experts (E, F, K), (E, F, K),
    (E, M, F) and the error bound of a binary32 computation whose products
    are exact: sums of n terms are off by (n + 64) EPS times the sum of
    magnitudes (the 64 covers the joining of partial sums), Swish'(z) is below
    1.1 in magnitude, and the epilogue rounds within 2^-20 of h."""
    N, M, F, K = x.shape[0], down.shape[1], gate.shape[1], gate.shape[2]
    y, bound = np.zeros((N, M)), np.full((N, M), 1e-30)
    for n in range(N):
        for s in range(ids.shape[1]):
            e = ids[n, s]
            if e < 0 or e >= gate.shape[0]:
                continue
            g, u = gate[e] @ x[n], up[e] @ x[n]
            eg = (K + 64) * EPS * (np.abs(gate[e]) @ np.abs(x[n]))
            eu = (K + 64) * EPS * (np.abs(up[e]) @ np.abs(x[n]))
            h = swish(g) * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(swish(g)) * eu + 2.0 ** -20 * np.abs(h)
            p = float(weights[n, s])
            y[n] += p * (down[e] @ h)
            # the terms of all of a token's experts join in one sum
            a = np.abs(down[e]) @ np.abs(h)
            bound[n] += abs(p) * (np.abs(down[e]) @ eh + (F * ids.shape[1] + 64) * EPS * a)
    return y, bound
