"""Products whose weights each token picks: grouped experts and adapters.

Each case is one call path of an inference engine over block-quantized weights
that serves prompts and many requests at once.  ``run`` computes it either in
plain torch operations (``own`` false) or with libqmm (``own`` true), on the
state that ``prepare`` made from a seed.

  group    slots (token, choice) in the order of their experts: the experts'
           first rows, the slots in that order, and each slot's place in it
  product  y[r] = W_e x[t(r)] for the rows r of each expert e, ragged
  swiglu   h[r] = Swish(Wg_e x[t(r)]) * (Wu_e x[t(r)]), likewise
  layer    y[n] = sum_s p[n][s] Wd_e h_e(x[n]), e = ids[n][s]: the three together
  lora     y[n] = base[n] + s_a B_a (A_a x[n]), a = ids[n]: each request's own
           low-rank adapter beside the projection that all share

Weight rows are 32- or 64-weight blocks: the blocks' scales (fp16, or for MXFP4
one power-of-two byte), zeros up to a multiple of 16 bytes, then the codes
(one signed byte each, or for the 4-bit types 16 bytes per 32 weights, byte j
= code j | code j+16 << 4).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
KINDS = ("q4_0", "q8_0", "mxfp4", "q4_b64", "q8_b64")


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # sixteen sequences decode together, two of eight experts each
        {"name": "group_16", "op": "group", "N": 16, "E": 8, "k": 2, "holes": False},
        # the tokens of several prompts, eight of 128 experts each, some slots empty
        {"name": "group_prompt", "op": "group", "N": 4093, "E": 128, "k": 8, "holes": True},
        # sixty-one sequences decode together: the down products of a small layer, about eight rows an expert
        {"name": "product_61", "op": "product", "type": "q4_b64", "N": 61, "E": 16, "k": 2, "K": 1408, "M": 2048,
         "gather": False, "out": "f32"},
        # a long prompt's down products, a thousand rows an expert
        {"name": "product_prompt", "op": "product", "type": "q8_0", "N": 4093, "E": 8, "k": 2, "K": 5632, "M": 2048,
         "gather": False, "out": "f32"},
        # thirty-three sequences over experts of four-bit floats
        {"name": "swiglu_33", "op": "swiglu", "type": "mxfp4", "N": 33, "E": 32, "k": 4, "K": 2048, "M": 1408,
         "gather": True, "out": "bf16"},
        # a 512-token prompt's gate and up products, two of eight large experts
        {"name": "swiglu_512", "op": "swiglu", "type": "q4_0", "N": 512, "E": 8, "k": 2, "K": 2048, "M": 5632,
         "gather": True, "out": "bf16"},
        # sixty-four sequences through a whole layer of many small experts
        {"name": "layer_64", "op": "layer", "type": "mxfp4", "N": 64, "E": 64, "k": 8, "K": 2048, "M": 1024,
         "holes": False},
        # a whole layer for the prompts of several requests, slots left empty at its capacity
        {"name": "layer_prompt", "op": "layer", "type": "q4_0", "N": 4096, "E": 8, "k": 2, "K": 2048, "M": 5632,
         "holes": True},
        # one sequence decodes with its adapter
        {"name": "lora_1", "op": "lora", "N": 1, "L": 4, "r": 16, "K": 2048, "M": 2048, "x": "f32", "base": True,
         "runs": False},
        # sixty-four requests decode, each token with one of twenty-four adapters or none
        {"name": "lora_64", "op": "lora", "N": 64, "L": 24, "r": 16, "K": 2048, "M": 5632, "x": "f32", "base": True,
         "runs": False},
        # seven requests' prompts, one adapter each
        {"name": "lora_prompt", "op": "lora", "N": 4093, "L": 7, "r": 64, "K": 2048, "M": 2048, "x": "bf16",
         "base": True, "runs": True},
        # the same through the wide projection, with a high rank and the adapters' part alone
        {"name": "lora_wide", "op": "lora", "N": 1021, "L": 3, "r": 128, "K": 5632, "M": 2048, "x": "bf16",
         "base": False, "runs": True},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("group", "product", "product", "swiglu", "layer", "lora", "lora"))
    if op == "lora":
        few = rng.random() < 0.5
        N = _spread(rng, 1, 256) if few else _spread(rng, 64, 4096)
        return {"op": op, "N": N, "L": _spread(rng, 1, 48 if few else 8), "r": _spread(rng, 8, 128, 8),
                "K": _spread(rng, 256, 5632, 32), "M": _spread(rng, 64, 5632), "x": "f32" if few else "bf16",
                "base": rng.random() < 0.7, "runs": not few}
    N, E = _spread(rng, 9, 4096), _spread(rng, 2, 128 if op == "group" else 64)
    k = rng.randint(1, min(E, 8))
    if op == "group":
        return {"op": op, "N": N, "E": E, "k": k, "holes": rng.random() < 0.5}
    kind, K = rng.choice(KINDS), _spread(rng, 256, 4096, 64)
    if op == "layer":
        F = _spread(rng, 256, 4096, 64)
        E = max(2, min(E, (1 << 27) // (K * F)))
        k = min(k, E)
        N = max(9, min(N, (1 << 36) // (k * K * F)))
        return {"op": op, "type": kind, "N": N, "E": E, "k": k, "K": K, "M": F, "holes": rng.random() < 0.5}
    M = _spread(rng, 65, 5632)
    E = max(2, min(E, (1 << 28) // (K * M)))
    k = min(k, E)
    N = max(9, min(N, (1 << 36) // (k * K * M)))
    return {"op": op, "type": kind, "N": N, "E": E, "k": k, "K": K, "M": M, "gather": op == "swiglu" or rng.random() < 0.5,
            "out": "bf16" if op == "swiglu" else rng.choice(("f32", "bf16"))}


# ------------------------------------------------------------ packed rows

def _block(kind):
    return 64 if kind.endswith("b64") else 32


def _scale_bytes(kind, K):
    n = K // _block(kind) * (1 if kind == "mxfp4" else 2)
    return n, -(-n // 16) * 16


def _row_bytes(kind, K):
    return _scale_bytes(kind, K)[1] + (K if kind.startswith("q8") else K // 2)


def _pad16(t):
    return torch.nn.functional.pad(t, (0, -t.shape[-1] % 16))


def _nibbles(codes):
    """(..., blocks, B) four-bit codes -> (..., B / 2 * blocks) bytes, by runs of 32."""
    c = codes.to(torch.uint8).unflatten(-1, (-1, 32))
    return (c[..., :16] | (c[..., 16:] << 4)).flatten(-3)


def _pack(w, kind):
    """float32 (..., K) -> packed rows."""
    b = w.unflatten(-1, (-1, _block(kind)))
    amax = b.abs().amax(-1)
    if kind == "mxfp4":
        e = torch.where(amax == 0, -127, torch.frexp(amax)[1] - 3).clamp(-127, 127)
        mag = b.abs() * torch.exp2(-e.float()).unsqueeze(-1)
        code = torch.stack([(mag >= m) if i % 2 else (mag > m) for i, m in enumerate(MIDS)]).sum(0, dtype=torch.int32)
        return torch.cat((_pad16((e + 127).to(torch.uint8)), _nibbles(code + torch.where(torch.signbit(b), 8, 0))), -1)
    d = (amax / (8.0 if kind.startswith("q4") else 127.0)).half()
    df = d.float().unsqueeze(-1)
    q = torch.where(df > 0, b / torch.where(df > 0, df, 1.0), 0.0)
    q = torch.sign(q) * torch.floor(q.abs() + 0.5)
    scales = _pad16(d.unsqueeze(-1).view(torch.uint8).flatten(-2))
    if kind.startswith("q4"):
        return torch.cat((scales, _nibbles((q + 8).clamp(0, 15))), -1)
    return torch.cat((scales, q.clamp(-127, 127).to(torch.int8).view(torch.uint8).flatten(-2)), -1)


# ------------------------------------------------------------- plain forms

def _unpack(rows, kind, K):
    """Packed rows (..., bytes) -> float32 (..., K)."""
    ns, off = _scale_bytes(kind, K)
    s = rows[..., :ns].contiguous()
    if kind == "mxfp4":
        e = s.int()
        d = torch.where(e == 0, 2.0 ** -127, (e << 23).view(torch.float32))
    else:
        d = s.view(torch.float16).float()
    if kind.startswith("q8"):
        q = rows[..., off:off + K].contiguous().view(torch.int8).float()
    else:
        by = rows[..., off:off + K // 2].unflatten(-1, (-1, 16))
        c = torch.cat((by & 15, by >> 4), -1).flatten(-2)
        q = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=rows.device)[c.int()] if kind == "mxfp4" else c.float() - 8.0
    return (q.unflatten(-1, (-1, _block(kind))) * d.unsqueeze(-1)).flatten(-2)


def _plain_group(ids, E):
    flat = ids.flatten().long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True)[1]
    counts = torch.zeros(E + 2, dtype=torch.int64, device=ids.device).index_add_(0, key + 1, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0)[:E + 1]
    at = torch.empty_like(order)
    at[order] = torch.arange(order.numel(), device=ids.device)
    return offsets.int(), order.int(), torch.where(key < E, at, -1).int().view(ids.shape)


def _padded(rows, offsets, cap):
    """The experts' rows side by side, (E, cap, K) in float32 with zeros after
    each expert's last one, and where row r of the grouped order went."""
    E, R = offsets.numel() - 1, rows.shape[0]
    first, count = offsets[:-1].long(), (offsets[1:] - offsets[:-1]).long()
    c = torch.arange(cap, device=rows.device)
    at = (first.unsqueeze(1) + c).clamp(max=max(R - 1, 0))
    x = torch.where((c < count.unsqueeze(1)).unsqueeze(-1), rows[at].float(), 0.0)
    r = torch.arange(R, device=rows.device)
    e = torch.searchsorted(offsets[1:].long().contiguous(), r, right=True).clamp(max=E - 1)
    return x, e * cap + (r - first[e]).clamp(0, cap - 1)


def _by_expert(x, w):
    """(E, cap, K) x (E, M, K) -> (E * cap, M)."""
    return torch.matmul(x, w.transpose(1, 2).contiguous()).flatten(0, 1)


def _swiglu(g, u):
    return g / (1.0 + torch.exp(-g)) * u


def _plain_products(s):
    rows = s["x"][s["order"].long() // s["k"]] if s["gather"] else s["x"]
    x, where = _padded(rows, s["offsets"], s["cap"])
    y = _by_expert(x, _unpack(s["w"], s["type"], s["K"]))
    if s["op"] == "swiglu":
        y = _swiglu(y, _by_expert(x, _unpack(s["up"], s["type"], s["K"])))
    return y[where].to(_DTYPE[s["out"]])


def _plain_layer(s):
    offsets, order, place = _plain_group(s["ids"], s["E"])
    x, where = _padded(s["x"][order.long() // s["k"]], offsets, s["cap"])
    h = _swiglu(_by_expert(x, _unpack(s["w"], s["type"], s["K"])), _by_expert(x, _unpack(s["up"], s["type"], s["K"])))
    d = _by_expert(h.unflatten(0, (s["E"], -1)), _unpack(s["down"], s["type"], s["M"]))[where]
    live = (place >= 0).unsqueeze(-1)
    y = torch.where(live, d[place.clamp(min=0).long()] * s["p"].unsqueeze(-1), 0.0).sum(1)
    return y.bfloat16()


def _plain_lora(s):
    offsets, order, place = _plain_group(s["ids"], s["L"])
    x, where = _padded(s["x"][order.long()], offsets, s["cap"])
    u = _by_expert(x, s["a"].float())
    d = _by_expert(u.unflatten(0, (s["L"], -1)), s["b"].float()).unflatten(0, (s["L"], -1)) * s["scales"].view(-1, 1, 1)
    d = torch.where((place >= 0).unsqueeze(-1), d.flatten(0, 1)[where][place.clamp(min=0).long()], 0.0)
    return s["add"] + d if s["base"] else d


# -------------------------------------------------------------- inputs

_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _choices(g, N, E, k):
    """k different experts of E for each token, some experts more popular than others."""
    return torch.topk(_randn(g, N, E) + 0.5 * _randn(g, E), k, dim=-1)


def _most(ids, E):
    """The most rows that one expert gets: a program's capacity."""
    flat = ids.flatten()
    return max(1, int(torch.bincount(flat[flat >= 0].long(), minlength=E).max()))


def prepare(case, seed):
    g, s = torch.Generator(device=DEV).manual_seed(seed), dict(case)
    op, N = case["op"], case["N"]
    if op == "lora":
        L, r, K, M = (case[n] for n in ("L", "r", "K", "M"))
        s["a"], s["b"] = (_randn(g, L, r, K) * 0.02).bfloat16(), (_randn(g, L, M, r) * 0.02).bfloat16()
        s["scales"] = torch.rand(L, generator=g, device=DEV) * 1.5 + 0.5
        s["x"] = _randn(g, N, K).to(_DTYPE[case["x"]])
        if case["base"]:
            s["add"] = _randn(g, N, M)
        if case["runs"]:    # prompts stand one after the other
            cuts = torch.sort(torch.randint(0, N + 1, (L - 1,), generator=g, device=DEV))[0]
            s["ids"] = torch.searchsorted(cuts, torch.arange(N, device=DEV), right=True).int()
        else:
            s["ids"] = torch.randint(0, L, (N,), generator=g, device=DEV).int()
            if N >= 8:      # requests without an adapter
                s["ids"].masked_fill_(torch.rand(N, generator=g, device=DEV) < 0.2, -1)
        s["cap"] = _most(s["ids"], L)
        return s
    E, k = case["E"], case["k"]
    top, ids = _choices(g, N, E, k)
    s["ids"], s["p"] = ids.int(), torch.softmax(top, -1)
    if case.get("holes"):
        s["ids"].masked_fill_(torch.rand((N, k), generator=g, device=DEV) < 0.1, -1)
        s["p"].masked_fill_(s["ids"] < 0, 0.0)
    if op == "group":
        return s
    K, M, kind = case["K"], case["M"], case["type"]
    s["cap"] = _most(s["ids"], E)
    s["w"] = _pack(_randn(g, E, M, K) * 0.02, kind)
    if op != "product":
        s["up"] = _pack(_randn(g, E, M, K) * 0.02, kind)
    if op == "layer":
        s["down"] = _pack(_randn(g, E, K, M) * 0.02, kind)
        s["x"] = _randn(g, N, K).bfloat16()
        return s
    s["offsets"], s["order"], _ = _plain_group(s["ids"], E)
    s["x"] = _randn(g, N if case["gather"] else N * k, K).bfloat16()
    return s


def _own(s):
    import quantized_matmul_ggml_amd as Q
    op = s["op"]
    if op == "group":
        return Q.moe_group(s["ids"], s["E"])
    if op == "lora":
        return Q.lora(s["a"], s["b"], s["x"], s["ids"], scales=s["scales"], base=s["add"] if s["base"] else None)
    kind = {"q4_0": Q.Q4_0, "q8_0": Q.Q8_0, "mxfp4": Q.MXFP4, "q4_b64": Q.Q4_B64, "q8_b64": Q.Q8_B64}[s["type"]]
    w = Q.Experts(s["w"], kind, s["K"], s["M"])
    if op == "layer":
        up, down = Q.Experts(s["up"], kind, s["K"], s["M"]), Q.Experts(s["down"], kind, s["M"], s["K"])
        return Q.moe_gemm_swiglu(w, up, down, s["x"], s["ids"], s["p"], dtype=torch.bfloat16)
    pick = {"order": s["order"], "top_k": s["k"]} if s["gather"] else {}
    if op == "swiglu":
        return Q.gemm_grouped_swiglu(w, Q.Experts(s["up"], kind, s["K"], s["M"]), s["x"], s["offsets"],
                                     dtype=_DTYPE[s["out"]], **pick)
    return Q.gemm_grouped(w, s["x"], s["offsets"], dtype=_DTYPE[s["out"]], **pick)


def run(s):
    if own:
        return _own(s)
    if s["op"] == "group":
        return _plain_group(s["ids"], s["E"])
    if s["op"] == "lora":
        return _plain_lora(s)
    return _plain_layer(s) if s["op"] == "layer" else _plain_products(s)


# ----------------------------------------------------------- work, 64 bits

def work(case):
    op, N = case["op"], case["N"]
    if op == "lora":
        L, r, K, M = (case[n] for n in ("L", "r", "K", "M"))
        with_one = N if case["runs"] or N < 8 else 0.8 * N
        used = min(L, N) if case["runs"] else L * (1.0 - (1.0 - 1.0 / L) ** with_one)
        x = K * (2 if case["x"] == "bf16" else 4)
        return {"bytes": int(used * 2 * r * (K + M) + with_one * x + N * M * (8 if case["base"] else 4)),
                "flops": int(2 * with_one * r * (K + M))}
    E, k = case["E"], case["k"]
    live = 0.9 if case.get("holes") else 1.0
    if op == "group":
        return {"bytes": 12 * N * k + 4 * (E + 1), "flops": 0}
    K, M, kind = case["K"], case["M"], case["type"]
    used = E * (1.0 - (1.0 - live * k / E) ** N)
    rows = live * N * k
    if op == "layer":
        one = 2 * M * _row_bytes(kind, K) + K * _row_bytes(kind, M)
        return {"bytes": int(used * one) + N * (4 * K + 8 * k), "flops": int(6 * rows * K * M)}
    many = 2 if op == "swiglu" else 1
    xs = (N if case["gather"] else N * k) * K * 2
    return {"bytes": int(used * many * M * _row_bytes(kind, K)) + xs + N * k * M * (2 if case["out"] == "bf16" else 4),
            "flops": int(2 * many * rows * K * M)}


def _values64(rows, kind, K):
    """Packed rows (R, bytes) -> float64 (R, K), each value worked out from its bits."""
    ns, off = _scale_bytes(kind, K)
    if kind == "mxfp4":
        d = torch.exp2(rows[:, :ns].double() - 127.0)
    else:
        h = rows[:, :ns:2].long() + 256 * rows[:, 1:ns:2].long()
        ex, m = (h >> 10) & 31, (h & 1023).double()
        d = torch.where(ex == 0, m * 2.0 ** -24, (1024.0 + m) * torch.exp2(ex.double() - 25.0))
    b = rows[:, off:]
    if kind.startswith("q8"):
        v = b[:, :K].double()
        q = torch.where(v > 127, v - 256.0, v)
    else:
        n = b[:, :K // 2].reshape(rows.shape[0], -1, 16)
        n = torch.stack((n % 16, n // 16), 2).reshape(rows.shape[0], K)
        if kind == "mxfp4":
            ex, m = ((n // 2) % 4).double(), (n % 2).double()
            q = torch.where(ex == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(ex - 1.0)) * (1.0 - 2.0 * (n // 8).double())
        else:
            q = n.double() - 8.0
    return (q.reshape(rows.shape[0], -1, _block(kind)) * d.unsqueeze(-1)).reshape(rows.shape[0], K)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "group":
        ids, E = s["ids"].cpu().numpy().ravel(), case["E"]
        runs = [np.flatnonzero(ids == e) for e in range(E)] + [np.flatnonzero((ids < 0) | (ids >= E))]
        place = np.full(ids.size, -1, np.int32)
        live = np.concatenate(runs[:E])
        place[live] = np.arange(live.size)
        return (np.cumsum([0] + [r.size for r in runs[:E]]).astype(np.int32), np.concatenate(runs).astype(np.int32),
                place.reshape(s["ids"].shape))
    x = s["x"].double()
    if op == "lora":
        y = s["add"].double() if case["base"] else torch.zeros((case["N"], case["M"]), dtype=torch.float64, device=DEV)
        for a in sorted(set(s["ids"].tolist()) - {-1}):
            rows = torch.nonzero(s["ids"] == a)[:, 0]
            y[rows] += float(s["scales"][a]) * (x[rows] @ s["a"][a].double().t() @ s["b"][a].double().t())
        return y
    ids, K, kind = s["ids"].cpu().numpy(), case["K"], case["type"]
    values = lambda name, e, C: _values64(s[name][e], kind, C).t()  # noqa: E731
    if op == "layer":
        y = torch.zeros((case["N"], K), dtype=torch.float64, device=DEV)
    else:
        y = torch.zeros((case["N"] * case["k"], case["M"]), dtype=torch.float64, device=DEV)
    done = 0
    for e in range(case["E"]):
        n, slot = np.nonzero(ids == e)
        if not n.size:
            continue
        n, slot = torch.from_numpy(n).to(DEV), torch.from_numpy(slot).to(DEV)
        rows = x[done:done + n.numel()] if op == "product" and not case["gather"] else x[n]
        v = rows @ values("w", e, K)
        if op != "product":
            v = v / (1.0 + torch.exp(-v)) * (rows @ values("up", e, K))
        if op == "layer":
            y.index_add_(0, n, s["p"][n, slot].double().unsqueeze(1) * (v @ values("down", e, case["M"])))
        else:
            y[done:done + n.numel()] = v
        done += n.numel()
    return y
