"""Cases of the gated feed-forward block's products, their gradient, and the 8-bit floating-point products.

Each case is one pass as a program around the routed layer makes it. ``run`` computes it in
plain torch (``own`` false) or through the package's entry points (``own`` true); ``exact``
computes the definition in float64.

* ``glu``: both projections of a gated block, the activation and its product with the up branch:
  h[r] = act(gate) with up = x[token[r]] . w[e, :I]^T, gate = x[token[r]] . w[e, I:]^T for the rows r
  of group e, act(gate, up) = min(gate, L) sigmoid(alpha min(gate, L)) (clamp(up, -L, L) + beta); with
  "pre" the projections [up, gate] themselves too, which a training step keeps in the operands' type.
* ``glu_back``: the gradient of [up, gate] from the projections that were kept, and h once more for the
  down weights' gradient; through the down product (dh = dy . w[e], "down") or from a dh that is
  there already.
* ``fp8``: each 128 consecutive values of a row of x to E4M3 with a scale of their own, then the product
  with E4M3 weights that have a scale for each block of 128 x 128, dense or by each row's expert.
* ``fp8_glu``: the same quantiser, then the gated block over such weights.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PLAIN = {"limit": 0.0, "alpha": 1.0, "beta": 0.0}           # silu(gate) * up
CLAMPED = {"limit": 7.0, "alpha": 1.0, "beta": 0.0}         # the layer's clamped SwiGLU
SHIFTED = {"limit": 7.0, "alpha": 1.702, "beta": 1.0}       # its alpha / beta form


def listed():
    return [
        # a test-sized layer: what one call costs
        {"name": "glu tiny", "op": "glu", "dtype": "bf16", "out": "bf16", "T": 4, "k": 2, "E": 8, "I": 136, "K": 256, "gather": True, "pre": False, "skew": 0.0, **CLAMPED},
        # gated block of a decode step: nearly every row has an expert to itself, so weights stream
        {"name": "glu decode", "op": "glu", "dtype": "bf16", "out": "bf16", "T": 8, "k": 6, "E": 384, "I": 576, "K": 7168, "gather": True, "pre": False, "skew": 0.0, **CLAMPED},
        # few, well filled experts in a training step, which keeps the projections
        {"name": "glu training", "op": "glu", "dtype": "fp16", "out": "fp16", "T": 8191, "k": 2, "E": 8, "I": 2048, "K": 4096, "gather": True, "pre": True, "skew": 0.2, **PLAIN},
        # the expert that every token passes, in a prefill batch
        {"name": "glu shared", "op": "glu", "dtype": "bf16", "out": "bf16", "T": 4097, "k": 1, "E": 1, "I": 2304, "K": 7168, "gather": False, "pre": False, **SHIFTED},
        # the backward pass of a training step with unequal loads, through the down product
        {"name": "glu_back training", "op": "glu_back", "dtype": "bf16", "T": 2048, "k": 8, "E": 32, "I": 1024, "N": 6144, "down": True, "h": True, "skew": 0.5, **CLAMPED},
        # the same in a small batch, many of the experts without a row
        {"name": "glu_back small", "op": "glu_back", "dtype": "fp16", "T": 67, "k": 2, "E": 64, "I": 576, "N": 7168, "down": True, "h": False, "skew": 0.7, **PLAIN},
        # from a dh that another operator left, over many rows
        {"name": "glu_back rows", "op": "glu_back", "dtype": "bf16", "T": 8191, "k": 2, "E": 1, "I": 2048, "N": 0, "down": False, "h": True, **CLAMPED},
        # a dense up/gate product next to the experts: a decode step and a prefill batch
        {"name": "fp8 decode", "op": "fp8", "dtype": "bf16", "out": "bf16", "T": 8, "k": 1, "E": 1, "N": 4608, "K": 7168},
        {"name": "fp8 prefill", "op": "fp8", "dtype": "bf16", "out": "bf16", "T": 4097, "k": 1, "E": 1, "N": 4608, "K": 7168},
        # up/gate product of a prefill batch with 8-bit experts
        {"name": "fp8 experts", "op": "fp8", "dtype": "bf16", "out": "bf16", "T": 4096, "k": 6, "E": 384, "N": 1152, "K": 7168, "skew": 0.3},
        # gated block of 8-bit experts: a decode step, and a prefill batch over fewer and larger experts
        {"name": "fp8_glu decode", "op": "fp8_glu", "dtype": "bf16", "out": "bf16", "T": 8, "k": 6, "E": 384, "I": 576, "K": 7168, "skew": 0.0, **CLAMPED},
        {"name": "fp8_glu prefill", "op": "fp8_glu", "dtype": "fp16", "out": "fp16", "T": 2048, "k": 8, "E": 32, "I": 1024, "K": 6144, "skew": 0.5, **PLAIN},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


MOST_WEIGHTS = 384 * 1152 * 7168
MOST_PRODUCTS = 16382 * 4096 * 4096


def draw(rng):
    op = rng.choice(["glu", "glu", "glu_back", "glu_back", "fp8", "fp8", "fp8_glu"])
    dense = rng.random() < 0.3
    k = 1 if dense else rng.choice([1, 2, 4, 6, 8])
    down = op != "glu_back" or rng.random() < 0.7
    while True:
        E = 1 if dense else _log(rng, 2, 384)
        inner, outer = 8 * _log(rng, 8, 512), 16 * _log(rng, 4, 448)
        T = _log(rng, 1, 8192 if dense else 16384 // k)
        width = inner if op in ("fp8", "glu_back") else 2 * inner
        if E * width * outer <= MOST_WEIGHTS and T * k * width * outer <= MOST_PRODUCTS:
            break
    dtype = rng.choice(["bf16", "fp16"])
    case = {"op": op, "dtype": dtype, "T": T, "k": k, "E": E, "skew": 0.0 if dense else rng.choice([0.0, 0.3, 0.7])}
    if op == "fp8":
        case.update(N=inner, K=outer)
    elif op == "glu_back":
        case.update(I=inner, N=outer if down else 0, down=down, h=rng.random() < 0.5)
    else:
        case.update(I=inner, K=outer)
    if op != "fp8":
        case.update(rng.choice([PLAIN, CLAMPED, SHIFTED]))
    if op != "glu_back":
        case["out"] = rng.choice([dtype, dtype, "fp32"])
    if op == "glu":
        case.update(gather=not dense and rng.random() < 0.5, pre=rng.random() < 0.5)
    return case


def _shares(case, device="cpu"):
    """The experts' shares of the routes: rank^-skew, in expert order."""
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -case.get("skew", 0.0)
    return (p / p.sum()).to(device)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, k, E, op = case["T"], case["k"], case["E"], case["op"]
    R, dt = T * k, DTYPES[case["dtype"]]
    s = dict(case)

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)

    s["first"] = s["token"] = None
    s["most"] = R
    if E > 1:
        # routes drawn by the experts' shares, sorted by expert in route order; the expert order is shuffled
        shares = _shares(case, "cuda")[torch.randperm(E, device="cuda", generator=g)]
        e = torch.multinomial(shares, R, replacement=True, generator=g)
        order = torch.argsort(e, stable=True)
        counts = torch.bincount(e, minlength=E)
        s["first"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        if op.startswith("fp8") or case.get("gather"):
            s["token"] = (order // k).to(torch.int32)
    if op == "glu_back":
        I, N = case["I"], case["N"]
        s["pre"] = normal(R, 2 * I, scale=2.0)     # projections wide enough that some meet the limit
        if case["down"]:
            s["dy"] = normal(R, N)
            s["w"] = normal(E, N, I, scale=1 / math.sqrt(N))
        else:
            s["dh"] = normal(R, I)
        return s
    K = case["K"]
    N = case["N"] if op == "fp8" else 2 * case["I"]
    if op == "glu":
        s["x"] = normal(R if s["token"] is None else T, K)
        s["w"] = normal(E, N, K, scale=2 / math.sqrt(K))
        return s
    x = normal(T if s["token"] is not None else R, K)
    x[:, torch.randperm(K, device="cuda", generator=g)[:max(1, K // 512)]] *= 12   # outlier channels
    s["x"] = x
    # weights as a checkpoint holds them: codes that fill E4M3's range, a scale a block of 128 x 128 (of each
    # branch of the gated block for itself)
    s["w"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        s["w"][e] = normal(N, K, scale=110.0, dtype=torch.float32).clamp_(-448, 448)
    kb, nb = -(-K // 128), -(-(N if op == "fp8" else N // 2) // 128)
    shape = (E, nb, kb) if op == "fp8" else (E, 2, nb, kb)
    s["w_scale"] = torch.empty(*shape, device="cuda").uniform_(0.5, 2.0, generator=g) / (110 * math.sqrt(K))
    return s


# ---------------------------------------------------------------- plain forms


def _padded(rows, first, most):
    """The rows of each group in a [E, most, ...] block padded with zeros, and where each row went."""
    if first is None:
        return rows[None], torch.arange(rows.shape[0], device=rows.device)
    E = first.numel() - 1
    r = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(first[1:].long(), r, right=True)
    at = e * most + r - first.long()[e]
    block = rows.new_zeros(E * most, rows.shape[1]).index_copy(0, at, rows)
    return block.view(E, most, -1), at


def _rows(x, token):
    return x if token is None else x[token.long()]


def _product(x, w, first, most):
    """x[r] . w[e]^T in 32 bits."""
    xp, at = _padded(x, first, most)
    return torch.bmm(xp, w.transpose(1, 2)).flatten(0, 1)[at]


def _branches(pre, s):
    """(up, gate) after the limit, and where the limit lets gradients through."""
    up, gate = pre.chunk(2, dim=1)
    if not s["limit"] > 0:
        return up, gate, None, None
    L = s["limit"]
    return up.clamp(-L, L), gate.clamp(max=L), up.abs() <= L, gate <= L


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v))


def _act(pre, s):
    up, gate, _, _ = _branches(pre, s)
    return gate * _sigmoid(s["alpha"] * gate) * (up + s["beta"])


def _act_back(dh, pre, s):
    up, gate, up_in, gate_in = _branches(pre, s)
    sig = _sigmoid(s["alpha"] * gate)
    d_up = dh * gate * sig
    d_gate = dh * (up + s["beta"]) * sig * (1 + s["alpha"] * gate * (1 - sig))
    if up_in is not None:
        d_up, d_gate = torch.where(up_in, d_up, 0.0), torch.where(gate_in, d_gate, 0.0)
    return torch.cat([d_up, d_gate], dim=1), gate * sig * (up + s["beta"])


def _quantise(x):
    """E4M3 codes and scales of 128 values each: scale = amax / 448, codes = x * (448 / amax), each rounded to 32
    bits (the quotients through 64: torch divides by and into a number through its reciprocal)."""
    kb = -(-x.shape[1] // 128)
    v = torch.nn.functional.pad(x.float(), (0, kb * 128 - x.shape[1])).view(x.shape[0], kb, 128)
    amax = v.abs().amax(2, keepdim=True)
    factor = torch.where(amax > 0, 448 / amax.double(), 0.0).float()
    codes = (v * factor).to(torch.float8_e4m3fn).float()
    return codes, (amax.double() / 448).float()


def _dequantised_weights(w, scale, branches):
    E, N, K = w.shape
    s = scale.repeat_interleave(128, -1)[..., :K]
    s = s.repeat_interleave(128, -2)[..., :N // branches, :]
    return w.float() * s.reshape(E, N, K)


def _plain(s):
    op = s["op"]
    if op == "glu_back":
        dt = s["pre"].dtype
        if s["down"]:
            dyp, at = _padded(s["dy"].float(), s["first"], s["most"])
            dh = torch.bmm(dyp, s["w"].float()).flatten(0, 1)[at]
        else:
            dh = s["dh"].float()
        d_pre, h = _act_back(dh, s["pre"].float(), s)
        return (d_pre.to(dt), h.to(dt)) if s["h"] else d_pre.to(dt)
    out = DTYPES[s["out"]]
    if op == "glu":
        pre = _product(_rows(s["x"], s["token"]).float(), s["w"].float(), s["first"], s["most"])
        h = _act(pre, s).to(out)
        return (h, pre.to(s["x"].dtype)) if s["pre"] else h
    codes, scale = _quantise(s["x"])
    x = (codes * scale).flatten(1)[:, :s["K"]]
    w = _dequantised_weights(s["w"], s["w_scale"], 1 if op == "fp8" else 2)
    y = _product(_rows(x, s["token"]), w, s["first"], s["most"])
    return (y if op == "fp8" else _act(y, s)).to(out)


def _framework(s):
    import block_scaled_fp4_histogram_amd as M

    op, first = s["op"], s["first"]
    form = {} if op == "fp8" else {"limit": s["limit"], "alpha": s["alpha"], "beta": s["beta"]}
    if op == "glu_back":
        if not s["down"]:
            return M.glu_grad(s["dh"], s["pre"], keep_h=s["h"], **form)
        if first is None:
            return M.glu_dx(s["dy"], s["w"][0], s["pre"], keep_h=s["h"], **form)
        return M.grouped_glu_dx(s["dy"], s["w"], s["pre"], first, keep_h=s["h"], **form)
    out = DTYPES[s["out"]]
    if op == "glu":
        if first is None:
            return M.glu(s["x"], s["w"][0], keep_pre=s["pre"], out_dtype=out, **form)
        return M.grouped_glu(s["x"], s["w"], first, rows=s["token"], keep_pre=s["pre"], out_dtype=out, **form)
    codes, scale = M.quant_fp8(s["x"])
    if op == "fp8":
        if first is None:
            return M.fp8_mm(codes, scale, s["w"][0], s["w_scale"][0], out_dtype=out)
        return M.grouped_fp8_mm(codes, scale, s["w"], s["w_scale"], first, rows=s["token"], out_dtype=out)
    if first is None:
        return M.fp8_glu(codes, scale, s["w"][0], s["w_scale"][0], out_dtype=out, **form)
    return M.grouped_fp8_glu(codes, scale, s["w"], s["w_scale"], first, rows=s["token"], out_dtype=out, **form)


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---------------------------------------------------------------- what a pass needs


def _size(name):
    return {"bf16": 2, "fp16": 2, "fp32": 4}[name]


def work(case):
    T, k, E, op = case["T"], case["k"], case["E"], case["op"]
    R, item = T * k, _size(case["dtype"])
    # experts that at least one of the R routes is expected to reach
    used = float((1 - (1 - _shares(case)) ** R).sum())
    if op == "glu_back":
        I, N = case["I"], case["N"]
        rows = R * I * item * (5 if case["h"] else 4)           # projections, their gradient, h
        if not case["down"]:
            return {"bytes": rows + R * I * item, "flops": 0}
        return {"bytes": rows + R * N * item + used * N * I * item, "flops": 2 * R * N * I}
    K, out = case["K"], _size(case["out"])
    N = case["N"] if op == "fp8" else 2 * case["I"]
    written = R * (N if op == "fp8" else N // 2) * out
    if op == "glu":
        x = T * K * item + 4 * R if case["gather"] else R * K * item
        return {"bytes": x + used * N * K * item + written + (R * N * item if case["pre"] else 0), "flops": 2 * R * N * K}
    index = 4 * R if E > 1 else 0
    blocks = -(-N // 128) * -(-K // 128)
    return {"bytes": T * K * item + index + used * (N * K + 4 * blocks) + written, "flops": 2 * R * N * K}


# ---------------------------------------------------------------- the definitions in float64


def _exact_codes(x):
    """Nearest E4M3 value of the 32-bit product x * fp32(448 / amax), ties to even, and fp32(amax / 448)."""
    rows, K = x.shape
    codes, scales = torch.zeros(rows, K, dtype=torch.float64, device=x.device), []
    for c in range(0, K, 128):
        v = x[:, c:c + 128].double()
        amax = v.abs().max(dim=1, keepdim=True).values
        r = torch.where(amax > 0, (448 / amax).float().double(), 0.0)
        v = (v * r).float().double()
        _, e = torch.frexp(v)
        step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)   # three bits after the leading one
        codes[:, c:c + 128] = torch.round(v / step) * step
        scales.append((amax / 448).float().double())
    return codes, torch.cat(scales, dim=1)


def _exact_act(up, gate, s, dh=None):
    L = s["limit"] if s["limit"] > 0 else math.inf
    u, g = up.clamp(-L, L) + s["beta"], gate.clamp(max=L)
    sig = torch.sigmoid(s["alpha"] * g)
    h = g * sig * u
    if dh is None:
        return h
    d_gate = dh * u * (sig + s["alpha"] * g * sig * (1 - sig)) * (gate <= L)
    return torch.cat([dh * g * sig * (up.abs() <= L), d_gate], dim=1), h


def exact(case, seed):
    """Group by group over slices in float64."""
    s = prepare(case, seed)
    op, R = s["op"], s["T"] * s["k"]
    bounds = [0, R] if s["first"] is None else s["first"].tolist()
    token = torch.arange(R, device="cuda") if s["token"] is None else s["token"].long()
    if op.startswith("fp8"):
        codes, scales = _exact_codes(s["x"])
        x = codes * scales.repeat_interleave(128, dim=1)[:, :s["K"]]
    elif op == "glu":
        x = s["x"].double()
    parts = []
    for e in range(s["E"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        if op == "glu_back":
            dh = s["dy"][lo:hi].double() @ s["w"][e].double() if s["down"] else s["dh"][lo:hi].double()
            up, gate = s["pre"][lo:hi, :s["I"]].double(), s["pre"][lo:hi, s["I"]:].double()
            parts.append(_exact_act(up, gate, s, dh))
            continue
        w = s["w"][e].double()
        if op.startswith("fp8"):
            halves = []
            for half, scale in zip(w.chunk(2) if op == "fp8_glu" else [w], s["w_scale"][e] if op == "fp8_glu" else s["w_scale"][e:e + 1]):
                n, kk = torch.arange(half.shape[0], device="cuda") // 128, torch.arange(s["K"], device="cuda") // 128
                halves.append(half * scale.double()[n][:, kk])
            w = torch.cat(halves)
        y = x[token[lo:hi]] @ w.t()
        if op == "fp8":
            parts.append((y,))
        else:
            half = y.shape[1] // 2
            parts.append((_exact_act(y[:, :half], y[:, half:], s), y))
    outs = [torch.cat(p) for p in zip(*parts)]
    if op == "fp8":
        return outs[0]
    if op == "glu_back":
        return tuple(outs) if s["h"] else outs[0]
    return tuple(outs) if s.get("pre") else outs[0]
