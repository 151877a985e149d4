"""Cases of the ragged expert products, the 8-bit integer products and the grouping of routes.

Each case is one pass as a program around the routed layer makes it. ``run`` computes it in
plain torch (``own`` false) or through the package's entry points (``own`` true); ``exact``
computes the definition in float64.

* ``group``: top-k expert ids [T, k] -> the routes sorted by expert: offsets of the groups, the
  route and the token of each sorted row, and each route's sorted row (-1 where the id is no
  expert's).
* ``mm``: out[r] = x[token[r]] . w[e]^T for the rows r of group e; ``mm_dx``: dx[r] = dy[r] . w[e];
  ``mm_dw``: dw[e] = sum over the rows r of group e of dy[r] (outer) x[token[r]].
* ``int8``: each token's row of x to 8-bit integers with a scale of its own, then the integer
  product with weights that have a scale for each output channel; ``int8_grouped``: the same with
  the weights of each row's expert.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a decode step's routes (8 tokens, the last two padding) and those of a long prefill
        {"name": "group decode", "op": "group", "T": 8, "k": 6, "E": 384, "pad": 2, "skew": 0.0},
        {"name": "group prefill", "op": "group", "T": 16384, "k": 8, "E": 256, "pad": 100, "skew": 0.7},
        # a test-sized layer: what one call costs
        {"name": "mm tiny", "op": "mm", "dtype": "bf16", "out": "bf16", "T": 4, "k": 2, "E": 8, "N": 256, "K": 256, "gather": True, "skew": 0.0},
        # up/gate product of a decode step: nearly every row has an expert to itself, so weights stream
        {"name": "mm decode", "op": "mm", "dtype": "bf16", "out": "bf16", "T": 8, "k": 6, "E": 384, "N": 1152, "K": 7168, "gather": True, "skew": 0.0},
        # up/gate product of a prefill batch over all experts, about 64 rows each
        {"name": "mm prefill", "op": "mm", "dtype": "bf16", "out": "bf16", "T": 4096, "k": 6, "E": 384, "N": 1152, "K": 7168, "gather": True, "skew": 0.3},
        # few, well filled experts, as a training step has them
        {"name": "mm training", "op": "mm", "dtype": "fp16", "out": "fp16", "T": 8191, "k": 2, "E": 8, "N": 4096, "K": 4096, "gather": False, "skew": 0.2},
        # its gradient for the rows, with unequal loads
        {"name": "mm_dx training", "op": "mm_dx", "dtype": "bf16", "out": "bf16", "T": 2048, "k": 8, "E": 32, "N": 1024, "K": 6144, "gather": False, "skew": 0.5},
        # its gradient for the weights, kept in 32 bits as optimisers want it
        {"name": "mm_dw training", "op": "mm_dw", "dtype": "bf16", "out": "fp32", "T": 2048, "k": 8, "E": 32, "N": 1024, "K": 6144, "gather": True, "skew": 0.5},
        # a down product's weight gradient in a small batch: short sums, many of the groups empty
        {"name": "mm_dw small", "op": "mm_dw", "dtype": "fp16", "out": "fp16", "T": 67, "k": 2, "E": 64, "N": 7168, "K": 576, "gather": False, "skew": 0.7},
        # a dense up/gate product next to the experts: a decode step and a prefill batch
        {"name": "int8 decode", "op": "int8", "dtype": "bf16", "out": "bf16", "T": 8, "k": 1, "E": 1, "N": 4608, "K": 7168},
        {"name": "int8 prefill", "op": "int8", "dtype": "bf16", "out": "bf16", "T": 4097, "k": 1, "E": 1, "N": 4608, "K": 7168},
        # up/gate product of a prefill batch with 8-bit experts
        {"name": "int8_grouped prefill", "op": "int8_grouped", "dtype": "bf16", "out": "bf16", "T": 4096, "k": 6, "E": 384, "N": 1152, "K": 7168, "skew": 0.3},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


MOST_WEIGHTS = 384 * 1152 * 7168
MOST_PRODUCTS = 16382 * 4096 * 4096


def draw(rng):
    op = rng.choice(["group", "mm", "mm", "mm_dx", "mm_dw", "int8", "int8_grouped"])
    k = rng.choice([1, 2, 4, 6, 8])
    if op == "group":
        T = _log(rng, 1, 16384)
        return {"op": op, "T": T, "k": k, "E": _log(rng, max(8, k), 512), "pad": rng.choice([0, T // 10]), "skew": rng.choice([0.0, 0.5, 0.9])}
    dense = op == "int8"
    while True:
        E = 1 if dense else _log(rng, 2, 384)
        N, K = 16 * _log(rng, 4, 448), 16 * _log(rng, 4, 448)
        T = _log(rng, 1, 8192 if dense else 16384 // k)
        if not dense:
            N = max(16, N - 8 * rng.choice([0, 1]))
        if E * N * K <= MOST_WEIGHTS and T * (1 if dense else k) * N * K <= MOST_PRODUCTS:
            break
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "T": T, "k": 1 if dense else k, "E": E, "N": N, "K": K}
    case["out"] = rng.choice([case["dtype"], "fp32"])
    if not dense:
        case["skew"] = rng.choice([0.0, 0.3, 0.7])
    if op in ("mm", "mm_dx", "mm_dw"):
        case["gather"] = op != "mm_dx" and rng.random() < 0.5
    return case


def _shares(case, device="cpu"):
    """The experts' shares of the routes: rank^-skew, in expert order."""
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -case.get("skew", 0.0)
    return (p / p.sum()).to(device)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, E = case["T"], case["k"], case["E"]
    s = dict(case)
    if case["op"] == "group":
        logits = torch.randn(T, E, device="cuda", generator=g) + torch.log(_shares(case, "cuda")).float()
        ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        if case["pad"]:
            ids[T - case["pad"]:] = -1
        s["ids"] = ids
        return s
    N, K, R, dt = case["N"], case["K"], T * k, DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)

    if case["op"] == "int8":
        s["first"] = s["token"] = None
    else:
        # routes drawn by the experts' shares, sorted by expert in route order; the expert order is shuffled
        shares = _shares(case, "cuda")[torch.randperm(E, device="cuda", generator=g)]
        e = torch.multinomial(shares, R, replacement=True, generator=g)
        order = torch.argsort(e, stable=True)
        counts = torch.bincount(e, minlength=E)
        s["first"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["token"] = (order // k).to(torch.int32)
        s["most"] = int(counts.max())
    if case["op"].startswith("int8"):
        x = normal(T, K)
        x[:, torch.randperm(K, device="cuda", generator=g)[:max(1, K // 512)]] *= 12   # outlier channels
        s["x"] = x
        s["w"] = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
        s["w_scale"] = torch.empty(E, N, device="cuda").uniform_(0.5, 2.0, generator=g) / (73 * math.sqrt(K))
        return s
    if case["op"] in ("mm", "mm_dx"):
        s["w"] = normal(E, N, K, scale=1 / math.sqrt(K if case["op"] == "mm" else N))
    if case["op"] in ("mm", "mm_dw"):
        s["x"] = normal(T if case["gather"] else R, K)
    if case["op"] in ("mm_dx", "mm_dw"):
        s["dy"] = normal(R, N)
    if not case.get("gather"):
        s["token"] = None
    return s


# ---------------------------------------------------------------- plain forms


def _group(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    keys, order = torch.sort(key, stable=True)
    first = torch.searchsorted(keys, torch.arange(E + 1, device=ids.device))
    at = torch.arange(T * k, device=ids.device)
    valid = at < first[E]
    inverse = torch.full_like(key, -1).scatter(0, order, torch.where(valid, at, -1))
    order = torch.where(valid, order, -1)
    token = torch.where(valid, order // k, -1)
    return first.to(torch.int32), order.to(torch.int32), token.to(torch.int32), inverse.view(T, k).to(torch.int32)


def _padded(rows, first, most):
    """The rows of each group in a [E, most, ...] block padded with zeros, and where each row went."""
    E = first.numel() - 1
    r = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(first[1:].long(), r, right=True)
    at = e * most + r - first.long()[e]
    block = rows.new_zeros(E * most, rows.shape[1]).index_copy(0, at, rows)
    return block.view(E, most, -1), at


def _rows(x, token):
    return x if token is None else x[token.long()]


def _mm(x, w, first, token, most, out):
    xp, at = _padded(_rows(x, token).float(), first, most)
    return torch.bmm(xp, w.float().transpose(1, 2)).flatten(0, 1)[at].to(out)


def _mm_dx(dy, w, first, most, out):
    dyp, at = _padded(dy.float(), first, most)
    return torch.bmm(dyp, w.float()).flatten(0, 1)[at].to(out)


def _mm_dw(dy, x, first, token, most, out):
    dyp, _ = _padded(dy.float(), first, most)
    xp, _ = _padded(_rows(x, token).float(), first, most)
    return torch.bmm(dyp.transpose(1, 2), xp).to(out)


def _quantise(x):
    """Row scale = largest magnitude / 127 in 32 bits; codes = x / scale to the nearest integer, in 64 bits (borders)."""
    scale = (x.double().abs().amax(1) / 127).float()
    codes = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[:, None]).clamp(-127, 127)
    return codes, scale


def _int8(x, w, w_scale, first, token, most, out):
    codes, scale = _quantise(x)   # codes as doubles: integer sums pass 2^24, exact in 64 bits
    if first is None:
        acc = codes @ w[0].double().t()
        return (acc.float() * scale[:, None] * w_scale).to(out)
    xp, at = _padded(codes[token.long()], first, most)
    acc = torch.bmm(xp, w.double().transpose(1, 2)).float() * w_scale[:, None, :]
    return (acc.flatten(0, 1)[at] * scale[token.long()][:, None]).to(out)


def _plain(s):
    op = s["op"]
    if op == "group":
        return _group(s["ids"], s["E"])
    out = DTYPES[s["out"]]
    if op == "mm":
        return _mm(s["x"], s["w"], s["first"], s["token"], s["most"], out)
    if op == "mm_dx":
        return _mm_dx(s["dy"], s["w"], s["first"], s["most"], out)
    if op == "mm_dw":
        return _mm_dw(s["dy"], s["x"], s["first"], s["token"], s["most"], out)
    return _int8(s["x"], s["w"], s["w_scale"], s["first"], s["token"], s.get("most"), out)


def _framework(s):
    import block_scaled_fp4_histogram_amd as M

    op = s["op"]
    if op == "group":
        return M.group_routes(s["ids"], s["E"])
    out = DTYPES[s["out"]]
    if op == "mm":
        return M.grouped_mm(s["x"], s["w"], s["first"], rows=s["token"], out_dtype=out)
    if op == "mm_dx":
        return M.grouped_mm_dx(s["dy"], s["w"], s["first"], out_dtype=out)
    if op == "mm_dw":
        return M.grouped_mm_dw(s["dy"], s["x"], s["first"], rows=s["token"], out_dtype=out)
    codes, scale = M.quant_int8(s["x"])
    if op == "int8":
        return M.int8_mm(codes, scale, s["w"][0], s["w_scale"][0], out_dtype=out)
    return M.grouped_int8_mm(codes, scale, s["w"], s["w_scale"], s["first"], rows=s["token"], out_dtype=out)


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------- what a pass needs


def _size(name):
    return {"bf16": 2, "fp16": 2, "fp32": 4}[name]


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if case["op"] == "group":
        return {"bytes": 4 * R + 4 * (E + 1) + 12 * R, "flops": 0}
    N, K, item, out = case["N"], case["K"], _size(case["dtype"]), _size(case["out"])
    # experts that at least one of the R routes is expected to reach
    used = float((1 - (1 - _shares(case)) ** R).sum())
    flops = 2 * R * N * K
    if case["op"] == "int8":
        return {"bytes": T * K * item + N * K + 4 * N + T * N * out, "flops": flops}
    if case["op"] == "int8_grouped":
        return {"bytes": T * K * item + used * (N * K + 4 * N) + 4 * R + R * N * out, "flops": flops}
    rows = T if case["gather"] else R
    x = rows * K * item + (4 * R if case["gather"] else 0)
    if case["op"] == "mm":
        return {"bytes": x + used * N * K * item + R * N * out, "flops": flops}
    if case["op"] == "mm_dx":
        return {"bytes": R * N * item + used * N * K * item + R * K * out, "flops": flops}
    return {"bytes": x + R * N * item + E * N * K * out, "flops": flops}


# ---------------------------------------------------------------- the definitions in float64


def exact(case, seed):
    """Group by group over slices in float64 (None for the routes' grouping, whose outputs are whole numbers)."""
    if case["op"] == "group":
        return None
    s = prepare(case, seed)
    op, E = s["op"], s["E"]
    if op.startswith("int8"):
        x = s["x"].double()
        scale = (x.abs().max(dim=1, keepdim=True).values / 127).float().double()   # a scale is a 32-bit value
        codes = torch.where(scale > 0, torch.round(x / scale), 0.0)
        if op == "int8":
            return (codes @ s["w"][0].double().t()) * scale * s["w_scale"][0].double()
    bounds = s["first"].tolist()
    R = bounds[-1]
    token = torch.arange(R, device="cuda") if s["token"] is None else s["token"].long()
    if op == "mm_dw":
        res = torch.zeros(E, s["N"], s["K"], dtype=torch.float64, device="cuda")
    else:
        res = torch.empty(R, s["K"] if op == "mm_dx" else s["N"], dtype=torch.float64, device="cuda")
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        if op == "mm":
            res[lo:hi] = s["x"][token[lo:hi]].double() @ s["w"][e].double().t()
        elif op == "mm_dx":
            res[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
        elif op == "mm_dw":
            res[e] = s["dy"][lo:hi].double().t() @ s["x"][token[lo:hi]].double()
        else:
            t = token[lo:hi]
            res[lo:hi] = (codes[t] @ s["w"][e].double().t()) * scale[t] * s["w_scale"][e].double()
    return res
