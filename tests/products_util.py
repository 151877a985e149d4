"""References in float64 and error bounds of the ragged products, the integer
products and the route grouping."""
import torch

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def offsets(counts, start=0):
    f = [start]
    for c in counts:
        f.append(f[-1] + c)
    return torch.tensor(f, dtype=torch.int32)


def gather(x, rows):
    """Rows of x behind the product rows in float64; zeros for numbers outside x."""
    if rows is None:
        return x.double()
    ok = (rows >= 0) & (rows < x.shape[0])
    return torch.where(ok[:, None], x[rows.long().clamp(0, max(x.shape[0] - 1, 0))].double(), 0.0)


def groups(first, R):
    f = first.clamp(0, R).tolist()
    for e in range(len(f) - 1):
        yield e, f[e], max(f[e], f[e + 1])


def ref_mm(x, w, first, rows, R):
    """(result, sum of the terms' magnitudes, covered rows) in float64."""
    xd = gather(x, rows)
    out = torch.zeros(R, w.shape[1], dtype=torch.float64, device=x.device)
    mag, cov = torch.zeros_like(out), torch.zeros(R, dtype=torch.bool, device=x.device)
    for e, lo, hi in groups(first, R):
        wd = w[e].double().t().contiguous()
        out[lo:hi], mag[lo:hi], cov[lo:hi] = xd[lo:hi] @ wd, xd[lo:hi].abs() @ wd.abs(), True
    return out, mag, cov


def ref_dx(dy, w, first):
    out = torch.zeros(dy.shape[0], w.shape[2], dtype=torch.float64, device=dy.device)
    mag, cov = torch.zeros_like(out), torch.zeros(dy.shape[0], dtype=torch.bool, device=dy.device)
    for e, lo, hi in groups(first, dy.shape[0]):
        wd = w[e].double()
        out[lo:hi], mag[lo:hi], cov[lo:hi] = dy[lo:hi].double() @ wd, dy[lo:hi].double().abs() @ wd.abs(), True
    return out, mag, cov


def ref_dw(dy, x, first, rows):
    xd = gather(x, rows)
    E = first.numel() - 1
    out = torch.zeros(E, dy.shape[1], xd.shape[1], dtype=torch.float64, device=dy.device)
    mag = torch.zeros_like(out)
    for e, lo, hi in groups(first, dy.shape[0]):
        d = dy[lo:hi].double().t().contiguous()
        out[e], mag[e] = d @ xd[lo:hi], d.abs() @ xd[lo:hi].abs()
    return out, mag


def assert_product(got, ref, mag, terms, label=""):
    """Elementwise: a sum of `terms` fp32-rounded terms is within terms * 2^-24 * (sum of magnitudes)
    of the exact one whatever its order (one rounding a term and addition, of at most half a step,
    eps/2 = 2^-24 each); the output type adds half a step of the result (eps/2, and half the
    smallest subnormal)."""
    fi = torch.finfo(got.dtype)
    acc = (terms + 1) * 2.0 ** -24 * mag
    tol = acc + (fi.eps / 2) * (ref.abs() + acc) + fi.tiny * fi.eps / 2
    bad = ~((got.double() - ref).abs() <= tol)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: got "
                             f"{got.flatten()[i].item()}, want {ref.flatten()[i].item()} +- {tol.flatten()[i].item()}")


def ref_quant(x):
    """(codes, scales) by the definition: fp32(amax / 127), nearest integer of the exact quotient."""
    amax = x.double().abs().amax(1)
    scale = (amax / 127).float()
    q = torch.round(x.double() / torch.where(scale > 0, scale, 1.0).double()[:, None]).clamp(-127, 127)
    bad = ~torch.isfinite(amax)
    q[bad] = 0
    scale[bad] = float("nan")
    return q.to(torch.int8), scale


def ref_int8(xq, xs, w, ws, first, rows, R):
    """Exact integer sums and the scaled result in float64."""
    xd = gather(xq, rows)
    sd = gather(xs[:, None], rows)
    out = torch.zeros(R, w.shape[1], dtype=torch.float64, device=w.device)
    cov = torch.zeros(R, dtype=torch.bool, device=w.device)
    for e, lo, hi in groups(first, R):
        out[lo:hi] = (xd[lo:hi] @ w[e].double().t().contiguous()) * sd[lo:hi] * ws[e].double()
        cov[lo:hi] = True
    return out, cov


def assert_int8(got, ref, label=""):
    """The integer sum is exact; its conversion to fp32 and the two scales round three times
    (2^-24 each), the output type once (eps/2)."""
    fi = torch.finfo(got.dtype)
    tol = (3.01 * 2.0 ** -24 + fi.eps / 2) * ref.abs() * (1 + 2.0 ** -20) + fi.tiny * fi.eps / 2 + 2.0 ** -126
    bad = ~((got.double() - ref).abs() <= tol)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.numel()} outside"


def ref_group(ids, E):
    """(first, order, token, inverse) lists by a stable sort in Python."""
    T, k = ids.shape
    flat = ids.flatten().tolist()
    routes = sorted((r for r, e in enumerate(flat) if 0 <= e < E), key=lambda r: (flat[r], r))
    first = [0] * (E + 1)
    for r in routes:
        first[flat[r] + 1] += 1
    for e in range(E):
        first[e + 1] += first[e]
    pad = [-1] * (T * k - len(routes))
    inverse = [-1] * (T * k)
    for p, r in enumerate(routes):
        inverse[r] = p
    i32 = torch.int32
    return (torch.tensor(first, dtype=i32), torch.tensor(routes + pad, dtype=i32),
            torch.tensor([r // k for r in routes] + pad, dtype=i32), torch.tensor(inverse, dtype=i32).view(T, k))
