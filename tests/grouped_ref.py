"""Plain float64 references for the products whose weights each token picks
(numpy on the CPU, from the formulas in include/qmm.h; no code shared with the
library), and the error bounds of binary32 sums of exact products."""
import numpy as np

import mx_ref as R

BF16 = 2.0 ** -8        # half a step of bfloat16, relative


def group(ids, E):
    """(offsets, order, place) of qmm_moe_group, one expert after the other."""
    flat = ids.ravel()
    runs = [np.flatnonzero(flat == e) for e in range(E)]
    empty = np.flatnonzero((flat < 0) | (flat >= E))
    order = np.concatenate(runs + [empty]).astype(np.int32)
    place = np.full(flat.size, -1, np.int32)
    for pos, slot in enumerate(order[:flat.size - empty.size]):
        place[slot] = pos
    offsets = np.concatenate([[0], np.cumsum([r.size for r in runs])]).astype(np.int32)
    return offsets, order, place.reshape(ids.shape)


def product(w, x):
    """(y, bound): rows x times the matrix w (M, K).  A block's sum is scaled
    before it joins the others, one rounding each; with the K products' sums and
    the joining of partial sums that is at most (K + K / 16 + 64) roundings of
    the sum of magnitudes."""
    K = w.shape[1]
    return x @ w.T, (K + K / 16 + 64) * R.EPS * (np.abs(x) @ np.abs(w).T) + 1e-30


def swiglu(g, eg, u, eu):
    """(h, bound) from the two sums and their bounds: Swish' is below 1.1 in
    magnitude, the epilogue rounds within 2^-20 of h."""
    s = R.swish(g)
    h = s * u
    return h, 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -20 * np.abs(h)


def rounded(y, bound, bf16):
    """The bound with one rounding to bf16."""
    return bound + BF16 * (np.abs(y) + bound) if bf16 else bound


def grouped(ws, x, offsets, order, top_k, bf16):
    """(y, bound, rows): ws the dequantized experts (E, M, K), or gate and up; NaN
    in rows outside the groups, whose numbers are not in `rows`."""
    n = x.shape[0] if order is None else order.size
    E, M = ws[0].shape[:2]
    y, bound = np.full((n, M), np.nan), np.zeros((n, M))
    rows = []
    for e in range(E):
        r = np.arange(offsets[e], offsets[e + 1])
        if not r.size:
            continue
        rows.append(r)
        t = r if order is None else order[r] // top_k
        v, b = product(ws[0][e], x[t])
        if len(ws) == 2:
            v, b = swiglu(v, b, *product(ws[1][e], x[t]))
        y[r], bound[r] = v, rounded(v, b, bf16)
    return y, bound, np.concatenate(rows) if rows else np.zeros(0, int)


def layer(gate, up, down, x, ids, weights, bf16):
    """(y, bound): float64 layer; h is rounded to bf16 between the products."""
    N, M, E = x.shape[0], down.shape[1], gate.shape[0]
    y, bound = np.zeros((N, M)), np.full((N, M), 1e-30)
    for e in range(E):
        n, s = np.nonzero(ids == e)
        if not n.size:
            continue
        h, eh = swiglu(*product(gate[e], x[n]), *product(up[e], x[n]))
        eh = rounded(h, eh, True)
        d, ed = product(down[e], h)
        ed = ed + eh @ np.abs(down[e]).T * (1 + 2.0 ** -10)
        p = weights[n, s].astype(np.float64)[:, None]
        np.add.at(y, n, p * d)
        # the weighted sum over the slots: a rounding for each term and sum
        np.add.at(bound, n, np.abs(p) * (ed + (2 * ids.shape[1] + 2) * R.EPS * (np.abs(d) + ed)))
    return y, rounded(y, bound, bf16)


def lora(a, b, x, ids, scales, base):
    """(y, bound): u = A x by binary32 sums of exact products (cut in at most 64
    parts), times the scale, rounded; then the sum over the rank and base."""
    L, r, K = a.shape
    N, M = x.shape[0], b.shape[1]
    y = np.zeros((N, M)) if base is None else base.astype(np.float64)
    bound = np.full((N, M), 1e-30)
    for n in range(N):
        i = int(ids[n])
        if i < 0 or i >= L:
            continue
        s = 1.0 if scales is None else float(scales[i])
        u, mag = a[i] @ x[n], np.abs(a[i]) @ np.abs(x[n])
        # three parts per product of a binary32 x
        eu = (3 * K + 128) * R.EPS * mag
        d = b[i] @ (s * u)
        ed = np.abs(b[i]) @ (abs(s) * (eu + 2 * R.EPS * (np.abs(u) + eu))) + (3 * r + 16) * R.EPS * (np.abs(b[i]) @ np.abs(s * u))
        y[n] += d
        bound[n] += ed + 2 * R.EPS * (np.abs(y[n]) + np.abs(d) + ed)
    return y, bound
