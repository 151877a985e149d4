"""Edges of the ragged products on the GPU: scales at the ends of fp32's range, groups without rows,
versions of given outputs, exceptions, and every tile shape next to rows, columns and values that are
not its own. References in float64 (tests/products_util.py)."""
import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from products_util import (BF16, FP16, FP32, assert_int8, assert_product, offsets, ref_dw, ref_dx, ref_int8, ref_mm)

pytestmark = pytest.mark.gpu


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=BF16, scale=1.0):
    return torch.randn(*shape, device="cuda", generator=g).mul_(scale).to(dtype)


# ---- integer products: scales at the ends of fp32's range

# pairs of an x scale and a w scale whose product leaves fp32's normal range, or whose x scale times the sum
# does, while the result is a number of fp32 (or, at the last, passes it)
ROW_SCALES = [1e-22, 2.4e36, 1.0, 1e-37, 2.0 ** -149, 3e30, 1e-30, 0.0]
CHANNEL_SCALES = [1e-22, 200.0, 1e-30, 2.0 ** -149, 1e-3, 3e36, 1.0, 5e-16]


def assert_scaled(got, ref, label=""):
    """The integer sum is exact. Its conversion to fp32, the product of the scales' fractions and their
    product round three times (2^-24 each of the value, whatever the scales' exponents); applying the
    exponents rounds only below 2^-126 (half of 2^-149), the output type once (half a step, or half its
    smallest subnormal). Results past the type's range are infinite: a reference within 2^-6 of it
    either way is not compared."""
    fi = torch.finfo(got.dtype)
    tol = (3.01 * 2.0 ** -24 + fi.eps / 2) * (1 + 2.0 ** -20) * ref.abs() + fi.tiny * fi.eps / 2 + 2.0 ** -150
    past = ref.abs() > fi.max * (1 + 2.0 ** -6)
    near = ref.abs() > fi.max * (1 - 2.0 ** -6)
    ok = torch.where(past, got.double() == torch.sign(ref) * float("inf"), ((got.double() - ref).abs() <= tol) | near)
    bad = (~ok).flatten().nonzero()
    assert bad.numel() == 0, (f"{label}: {bad.numel()} of {ok.numel()} outside, first at {int(bad[0])}: got "
                              f"{got.flatten()[bad[0]].item()}, want {ref.flatten()[bad[0]].item()}")


@pytest.mark.parametrize("counts,K", [([5], 1040), ([3, 0, 8], 272), ([700, 0, 333], 272), ([90, 0, 140], 8192)])
@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
def test_int8_scales_at_the_ends_of_the_range(counts, K, out_dtype):
    """Streamed rows, tiles and split reductions: a result that the output type holds comes out whatever its
    scales' product does, and a zero sum is zero."""
    g = _gen(K)
    R, E, N = sum(counts), len(counts), 1032
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, w = i8(R, K), i8(E, N, K)
    x[1::5] = 0
    xs = torch.tensor(ROW_SCALES, device="cuda").repeat(R // 8 + 1)[:R].contiguous()
    ws = torch.tensor(CHANNEL_SCALES, device="cuda").repeat_interleave(3).repeat(N // 24)[:N].repeat(E, 1).contiguous()
    first = offsets(counts).cuda()
    ref, _ = ref_int8(x, xs, w, ws, first, None, R)
    assert bool((ref[1::5] == 0).all())
    assert_scaled(M.grouped_int8_mm(x, xs, w, ws, first, out_dtype=out_dtype), ref, "grouped")
    if E == 1:
        assert_scaled(M.int8_mm(x, xs, w[0], ws[0], out_dtype=out_dtype), ref, "dense")


def test_int8_products_of_a_row_near_the_largest_value():
    """A bf16 row of 3e38 has a scale of 2.4e36; orthogonal codes still give zeros with large channel scales."""
    x = torch.zeros(2, 32, dtype=BF16, device="cuda")
    x[0, :16], x[1, 16:] = 3e38, 1.0
    q, s = M.quant_int8(x)
    w = q.repeat(4, 1).contiguous()
    out = M.int8_mm(q, s, w, torch.full((8,), 4e3, device="cuda"), out_dtype=FP32)
    assert out[0, 1::2].tolist() == [0.0] * 4 and out[1, 0::2].tolist() == [0.0] * 4
    assert bool(torch.isinf(out[0, 0::2]).all())


@pytest.mark.parametrize("counts,N,K", [([0, 70, 0, 33], 136, 72), ([5000, 0, 3001], 72, 136)])
@pytest.mark.parametrize("gathered", [False, True])
def test_accumulating_leaves_groups_without_rows_bit_for_bit(counts, N, K, gathered):
    """Nothing is added there: negative zeros keep their sign, NaNs their bits (whole and split reductions)."""
    E, R = len(counts), sum(counts)
    g = _gen(N)
    dy, x = _normal(g, R, N), _normal(g, R, K)
    rows = torch.randperm(R, device="cuda", generator=g).to(torch.int32) if gathered else None
    base = torch.randn(E, N, K, device="cuda", generator=g)
    base[:, ::2, 1::3] = -0.0
    base[0, 1, 2] = base[1, 3, 4] = -float("nan")
    out = base.clone()
    first = offsets(counts).cuda()
    M.grouped_mm_dw(dy, x, first, rows=rows, out=out, accumulate=True)
    ref, mag = ref_dw(dy, x, first, rows)
    for e, c in enumerate(counts):
        if c == 0:
            assert torch.equal(out[e].view(torch.int32), base[e].view(torch.int32))
            continue
        fin = torch.isfinite(base[e])
        assert bool((torch.isfinite(out[e]) == fin).all())
        b = base[e].double()
        assert_product(out[e][fin], (ref[e] + b)[fin], (mag[e] + b.abs())[fin], c + 1)
    none = base.clone()
    M.grouped_mm_dw(dy[:0], x[:0], torch.zeros(E + 1, dtype=torch.int32, device="cuda"), out=none, accumulate=True)
    assert torch.equal(none.view(torch.int32), base.view(torch.int32))


def test_out_of_memory_keeps_its_type():
    """An output that no card holds (2 TiB): the allocator's own exception, and the next call works."""
    dy, first = torch.zeros(1, 1 << 20, dtype=BF16, device="cuda"), offsets([1]).cuda()
    with pytest.raises(torch.OutOfMemoryError):
        M.grouped_mm_dw(dy, dy, first)
    x = torch.ones(1, 8, dtype=BF16, device="cuda")
    assert M.grouped_mm_dw(x, x, first).tolist() == [[[1.0] * 8] * 8]


class _Product(torch.autograd.Function):
    """grouped_mm recorded by autograd, as a training program wraps it: rows in order, both gradients."""

    @staticmethod
    def forward(ctx, x, w, first):
        ctx.save_for_backward(x, w, first)
        return M.grouped_mm(x, w, first)

    @staticmethod
    def backward(ctx, dy):
        x, w, first = ctx.saved_tensors
        return M.grouped_mm_dx(dy, w, first), M.grouped_mm_dw(dy, x, first), None


def test_products_in_an_autograd_function():
    """Two products in a row through autograd: the gradients are the entry points', bit for bit, and the
    operands themselves are refused outside the function."""
    g = _gen(32)
    first = offsets([9, 0, 30, 1]).cuda()
    x, w1, w2 = (_normal(g, *s).requires_grad_() for s in ((40, 72), (4, 136, 72), (4, 24, 136)))
    dout = _normal(g, 40, 24)
    _Product.apply(_Product.apply(x, w1, first), w2, first).backward(dout)
    with torch.no_grad():
        h = M.grouped_mm(x, w1, first)
        dh = M.grouped_mm_dx(dout, w2, first)
        want = (M.grouped_mm_dx(dh, w1, first), M.grouped_mm_dw(dh, x, first), M.grouped_mm_dw(dout, h, first))
    for t, r in zip((x, w1, w2), want):
        assert torch.equal(t.grad, r)
    with pytest.raises(ValueError, match="x requires grad"):
        M.grouped_mm(x, w1, first)


def _written_outputs():
    """(name, given output, call into it) of every entry point that takes one."""
    g = _gen(31)
    x, w, dy, first = _normal(g, 6, 16), _normal(g, 2, 8, 16), _normal(g, 6, 8), offsets([2, 4]).cuda()
    q, s = M.quant_int8(x)
    wq, ws = M.quant_int8(w.view(16, 16))
    new = lambda *shape, dtype=BF16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
    o = [new(6, 8), new(6, 16), new(2, 8, 16, dtype=FP32), new(6, 16, dtype=torch.int8), new(6, dtype=FP32), new(6, 8), new(6, 8)]
    return [("grouped_mm", o[0], lambda t: M.grouped_mm(x, w, first, out=t)),
            ("grouped_mm_dx", o[1], lambda t: M.grouped_mm_dx(dy, w, first, out=t)),
            ("grouped_mm_dw", o[2], lambda t: M.grouped_mm_dw(dy, x, first, out=t, accumulate=True)),
            ("quant_int8", o[3], lambda t: M.quant_int8(x, out=t)),
            ("quant_int8 scales", o[4], lambda t: M.quant_int8(x, scales=t)),
            ("int8_mm", o[5], lambda t: M.int8_mm(q, s, wq[:8], ws[:8], out=t)),
            ("grouped_int8_mm", o[6], lambda t: M.grouped_int8_mm(q, s, wq.view(2, 8, 16), ws.view(2, 8), first, out=t))]


def test_given_outputs_advance_their_version():
    """As torch's own writes in place do, also where autograd is off or the output is an inference tensor."""
    for name, out, call in _written_outputs():
        for step in (1, 2):
            call(out)
            assert out._version == step, name
        with torch.no_grad():
            call(out)
        assert out._version == 3, name
        with torch.inference_mode():
            inf = torch.zeros_like(out)
            call(inf)
        call(inf)
        assert torch.equal(inf, out) or name == "grouped_mm_dw", name


def test_overwriting_a_saved_tensor_is_reported_by_backward():
    for name, out, call in _written_outputs():
        if not out.is_floating_point():
            continue
        p = torch.ones_like(out, requires_grad=True)
        loss = (out * p).sum()                        # saves out for p's gradient
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


# ---- every tile shape: sizes that select it, next to rows, columns and values that are not its own
#
# Reductions of more than two steps with a partial last one, columns past the last whole tile, groups of
# odd sizes and without rows, product rows in front of the groups and behind them. Infinities and NaNs stand
# in single operands' ends and in everything that no output may read; they have to reach the sums they are
# a term of and no other. (E, R, N, K, rows, columns of the tile, whether the reduction is split)

FORWARD = {"64x128": (5, 900, 1048, 200, 64, 128, False), "128x128": (5, 2900, 3080, 200, 128, 128, False),
           "128x256": (40, 5000, 4104, 136, 128, 256, False), "256x128": (5, 3000, 4104, 200, 256, 128, False),
           "split": (5, 400, 264, 4104, 64, 128, True), "stream": (5, 75, 264, 520, 16, 16, False),
           "130 groups": (130, 9000, 136, 200, 64, 128, False), "1000 groups": (1000, 9000, 264, 136, 64, 128, False),
           "split of 100 groups": (100, 6500, 72, 4104, 64, 128, True)}
DX = {"64x128": (5, 900, 200, 1048, 64, 128, False), "128x128": (5, 2900, 200, 3080, 128, 128, False),
      "128x256": (40, 5000, 136, 4104, 128, 256, False), "256x128": (5, 3000, 200, 4104, 256, 128, False),
      "split": (5, 300, 2600, 264, 64, 128, True), "130 groups": (130, 9000, 200, 136, 64, 128, False),
      "1000 groups": (1000, 9000, 136, 264, 64, 128, False), "split of 100 groups": (100, 6500, 4104, 72, 64, 128, True)}
DW = {"128x128": (8, 1200, 520, 1048, 128, 128, False), "256x128": (4, 1100, 2056, 1544, 256, 128, False),
      "split": (3, 8040, 72, 136, 128, 128, True), "1000 groups": (1000, 3000, 72, 40, 128, 128, False)}
INT8 = {"64x128": (5, 900, 1048, 400, 64, 128, False), "128x128": (5, 2900, 3080, 400, 128, 128, False),
        "128x256": (40, 5000, 4104, 272, 128, 256, False), "256x128": (5, 3000, 4104, 400, 256, 128, False),
        "split": (5, 400, 264, 8208, 64, 128, True), "stream": (5, 75, 264, 1040, 16, 16, False),
        "130 groups": (130, 9000, 136, 400, 64, 128, False), "1000 groups": (1000, 9000, 264, 272, 64, 128, False),
        "split of 100 groups": (100, 6500, 72, 8208, 64, 128, True)}
DENSE = {"64x128": (1, 900, 1048, 400, 64, 128, False), "128x128": (1, 2900, 3080, 400, 128, 128, False),
         "128x256": (1, 1876, 8200, 272, 128, 256, False), "256x128": (1, 3000, 4104, 400, 256, 128, False)}
START, TAIL = 3, 5


def _selected(op, case):
    """Operand sizes of a case, which have to select the shape it is named after."""
    E, R, N, K, rows, cols, split = case
    got = M.debug_mm_plan(op, E, R, N, K)
    assert got[:2] == (rows, cols) and (got[2] > 1) == split, got
    return E, R, N, K


def _ragged(E, R):
    """Group sizes of R - START - TAIL rows: the second group empty (where there are three), the last one a
    single row, the others uneven."""
    n = R - START - TAIL
    w = [1 + (5 * e) % 7 for e in range(E)]
    w[-1] = 0
    if E > 2:
        w[1] = 0
    counts = [(n - 1) * x // sum(w) for x in w]
    counts[-1] = 1
    counts[0] += n - sum(counts)
    return counts


def _numbered(g, R, T):
    """Row numbers: any row of x but its last inside the groups (two of them no row), the last one outside."""
    rows = torch.randint(0, T - 1, (R,), device="cuda", generator=g, dtype=torch.int32)
    rows[START + 1], rows[START + 6] = -1, T + 3
    rows[:START] = rows[R - TAIL:] = T - 1
    return rows


def _same_finite(got, ref):
    fin = torch.isfinite(ref)
    assert bool((torch.isfinite(got) == fin).all()) and not bool(fin.all()) and bool(fin.any())
    return fin


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", FORWARD)
def test_forward_tiles(shape, dtype, gathered):
    E, R, N, K = _selected(M.MM_FORWARD, FORWARD[shape])
    g = _gen(41)
    counts = _ragged(E, R)
    first = offsets(counts, START).cuda()
    T = R // 2 if gathered else R
    x, w = _normal(g, T, K, dtype=dtype), _normal(g, E, N, K, dtype=dtype)
    rows = _numbered(g, R, T) if gathered else None
    x[T - 1] = float("nan")
    if not gathered:
        x[:START], x[R - TAIL:] = float("nan"), float("inf")
    x[T // 3, K - 1], x[T // 3 + 1, 0], x[T // 2, K // 2] = float("inf"), float("nan"), float("-inf")
    w[0, N - 1, 0], w[0, 7, K - 1], w[1], w[2, 0, 0], w[E - 1, N // 2, K // 2] = (float("nan"),) * 5
    ref, mag, cov = ref_mm(x, w, first, rows, R)
    assert int(cov.sum()) == R - START - TAIL
    for out_dtype in (dtype, FP32):
        out = M.grouped_mm(x, w, first, rows=rows, out=torch.full((R, N), 7.5, dtype=out_dtype, device="cuda"))
        assert bool((out[~cov] == 7.5).all())
        fin = _same_finite(out[cov], ref[cov])
        assert_product(out[cov][fin], ref[cov][fin], mag[cov][fin], K, shape)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", DX)
def test_row_gradient_tiles(shape, dtype):
    E, R, N, K = _selected(M.MM_DX, DX[shape])
    g = _gen(42)
    first = offsets(_ragged(E, R), START).cuda()
    dy, w = _normal(g, R, N, dtype=dtype), _normal(g, E, N, K, dtype=dtype)
    dy[:START], dy[R - TAIL:] = float("nan"), float("inf")
    dy[R // 3, N - 1], dy[R // 3 + 1, 0], dy[R // 2, N // 2] = float("inf"), float("nan"), float("-inf")
    w[0, 0, K - 1], w[0, N - 1, 9], w[1], w[2, 0, 0], w[E - 1, N // 2, K // 2] = (float("nan"),) * 5
    ref, mag, cov = ref_dx(dy, w, first)
    for out_dtype in (dtype, FP32):
        out = M.grouped_mm_dx(dy, w, first, out=torch.full((R, K), 7.5, dtype=out_dtype, device="cuda"))
        assert bool((out[~cov] == 7.5).all())
        fin = _same_finite(out[cov], ref[cov])
        assert_product(out[cov][fin], ref[cov][fin], mag[cov][fin], N, shape)


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", DW)
def test_weight_gradient_tiles(shape, dtype, gathered):
    """Each group held to its own number of terms; accumulated, to one more."""
    E, R, N, K = _selected(M.MM_DW, DW[shape])
    g = _gen(43)
    counts = _ragged(E, R)
    first = offsets(counts, START).cuda()
    T = R // 2 if gathered else R
    dy, x = _normal(g, R, N, dtype=dtype), _normal(g, T, K, dtype=dtype)
    rows = _numbered(g, R, T) if gathered else None
    dy[:START], dy[R - TAIL:], x[T - 1] = float("nan"), float("inf"), float("nan")
    if not gathered:
        x[:START], x[R - TAIL:] = float("inf"), float("nan")
    last = START + counts[0] - 1                        # last row of the first group; the next begins behind it
    dy[last, N - 1], dy[last + 1, 3], dy[R - TAIL - 1, N // 2] = float("inf"), float("nan"), float("-inf")
    x[T // 3, K - 1], x[T // 3 + 1, 0] = float("nan"), float("inf")
    ref, mag = ref_dw(dy, x, first, rows)
    for out_dtype in (dtype, FP32):
        dw = M.grouped_mm_dw(dy, x, first, rows=rows, out_dtype=out_dtype)
        fin = _same_finite(dw, ref)
        for e, c in enumerate(counts):
            assert_product(dw[e][fin[e]], ref[e][fin[e]], mag[e][fin[e]], c, f"{shape}, group {e}")
    base = torch.randn(E, N, K, device="cuda", generator=g)
    dw = M.grouped_mm_dw(dy, x, first, rows=rows, out=base.clone(), accumulate=True)
    _same_finite(dw, ref)
    for e, c in enumerate(counts):
        b = base[e].double()
        assert_product(dw[e][fin[e]], (ref[e] + b)[fin[e]], (mag[e] + b.abs())[fin[e]], c + 1, f"{shape}, group {e}")


def _int8_operands(g, E, R, N, K, T):
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, w = i8(T, K), i8(E, N, K)
    xs, ws = torch.rand(T, device="cuda", generator=g) + 0.1, (torch.rand(E, N, device="cuda", generator=g) + 0.1) / K / 100
    xs[T // 3], xs[T // 2] = float("nan"), float("inf")
    ws[0, N - 1], ws[E - 1, 0] = float("nan"), float("inf")
    return x, xs, w, ws


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("shape", INT8)
def test_int8_tiles(shape, gathered):
    E, R, N, K = _selected(M.MM_INT8, INT8[shape])
    g = _gen(44)
    first = offsets(_ragged(E, R), START).cuda()
    T = R // 2 if gathered else R
    x, xs, w, ws = _int8_operands(g, E, R, N, K, T)
    rows = _numbered(g, R, T) if gathered else None
    xs[T - 1], ws[1] = float("nan"), float("nan")
    if not gathered:
        xs[:START] = xs[R - TAIL:] = float("nan")
    ref, cov = ref_int8(x, xs, w, ws, first, rows, R)
    for out_dtype in (BF16, FP16, FP32):
        out = M.grouped_int8_mm(x, xs, w, ws, first, rows=rows, out=torch.full((R, N), 7.5, dtype=out_dtype, device="cuda"))
        assert bool((out[~cov] == 7.5).all())
        fin = _same_finite(out[cov], ref[cov])
        assert_int8(out[cov][fin], ref[cov][fin], shape)


@pytest.mark.parametrize("shape", DENSE)
def test_dense_int8_tiles(shape):
    E, R, N, K = _selected(M.MM_INT8, DENSE[shape])
    x, xs, w, ws = _int8_operands(_gen(45), E, R, N, K, R)
    ref, _ = ref_int8(x, xs, w, ws, offsets([R]).cuda(), None, R)
    for out_dtype in (BF16, FP32):
        out = M.int8_mm(x, xs, w[0], ws[0], out_dtype=out_dtype)
        fin = _same_finite(out, ref)
        assert_int8(out[fin], ref[fin], shape)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", ["64x128", "128x128", "256x128"])
def test_one_group_tiles(shape, dtype):
    """A single group of all rows, forward and row gradient: the sizes of the tile shapes above."""
    R, N, K = FORWARD[shape][1:4]
    assert M.debug_mm_plan(M.MM_FORWARD, 1, R, N, K) == FORWARD[shape][4:6] + (1,)
    assert M.debug_mm_plan(M.MM_DX, 1, R, K, N) == FORWARD[shape][4:6] + (1,)
    g = _gen(46)
    first = offsets([R]).cuda()
    x, w = _normal(g, R, K, dtype=dtype), _normal(g, 1, N, K, dtype=dtype)
    ref, mag, _ = ref_mm(x, w, first, None, R)
    assert_product(M.grouped_mm(x, w, first), ref, mag, K, shape)
    wt = w.transpose(1, 2).contiguous()                 # the same product as a row gradient
    assert_product(M.grouped_mm_dx(x, wt, first), ref, mag, K, shape)


def test_exact_sums_in_each_shape():
    """Integers whose sums fp32 holds exactly: every shape gives the definition's values, twice."""
    g = _gen(47)
    for E, R, N, K, _, _, _ in FORWARD.values():
        ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).to(BF16)  # noqa: E731
        x, w, first = ints(R, K), ints(E, N, K), offsets(_ragged(E, R), START).cuda()
        out = M.grouped_mm(x, w, first, out_dtype=FP32)
        ref, _, cov = ref_mm(x, w, first, None, R)
        assert torch.equal(out[cov].double(), ref[cov])
        assert torch.equal(M.grouped_mm(x, w, first, out_dtype=FP32)[cov], out[cov])


# ---- rows past 4 GiB

def test_gathered_rows_past_4_gib():
    """Row numbers whose bytes begin past 2^32, in products of a few rows (streamed, and weight gradients) and
    of many (tiles). Values are integers up to 3 in magnitude and sums stay below 2^24, so results are exact in
    fp32 and compared with equality; the row that each number would name with its byte offset cut to 32 bits
    holds other values, whose result is not the same."""
    g = _gen(51)
    K, N = 4096, 72
    T = 530001                                        # x of 4.34e9 bytes
    x = torch.randint(-3, 4, (T, K), device="cuda", generator=g, dtype=torch.int8).to(BF16)
    wrapped = 2 ** 32 // (2 * K)                      # rows in 4 GiB
    for R in (7, 700):
        rows = torch.randint(wrapped + 1, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        rows[0], rows[-1] = T - 1, wrapped
        first = offsets([R - 3, 3]).cuda()
        ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).to(BF16)  # noqa: E731
        w, dy = ints(2, N, K), ints(R, N)
        far, near = x[rows.long()], x[rows.long() - wrapped]
        ref, other = (ref_mm(t, w, first, None, R)[0] for t in (far, near))
        assert bool((ref != other).any(1).all())      # a cut offset changes every row
        assert torch.equal(M.grouped_mm(x, w, first, rows=rows, out_dtype=FP32).double(), ref)
        ref, other = (ref_dw(dy, t, first, None)[0] for t in (far, near))
        assert bool((ref != other).flatten(1).any(1).all())
        assert torch.equal(M.grouped_mm_dw(dy, x, first, rows=rows, out_dtype=FP32).double(), ref)


def test_rows_in_order_past_4_gib():
    """The same without row numbers: groups at the end of an x, a dy and an output past 4 GiB."""
    g = _gen(52)
    K, N, R = 4096, 72, 530001
    big = torch.randint(-3, 4, (R, K), device="cuda", generator=g, dtype=torch.int8).to(BF16)
    ints = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).to(BF16)  # noqa: E731
    small, w = ints(R, N), ints(3, N, K)
    first = offsets([R - 307, 300, 7]).cuda()
    end, cut = slice(R - 307, R), offsets([0, 300, 7]).cuda()
    out = M.grouped_mm(big, w, first, out_dtype=FP32)
    assert torch.equal(out[end].double(), ref_mm(big[end], w, cut, None, 307)[0])
    dx = M.grouped_mm_dx(small, w, first)             # sums up to 648: bf16 rounds them, half a step each
    ref, mag, _ = ref_dx(small[end], w, cut)
    assert_product(dx[end], ref, mag, N)
    dw = M.grouped_mm_dw(small, big, first, out_dtype=FP32)
    assert torch.equal(dw[1:].double(), ref_dw(small[end], big[end], cut, None)[0][1:])
    wt = w.transpose(1, 2).contiguous()               # the forward product as a row gradient: a dy past 4 GiB
    dx = M.grouped_mm_dx(big, wt, first, out_dtype=FP32)
    assert torch.equal(dx[end].double(), ref_mm(big[end], w, cut, None, 307)[0])


def test_gathered_int8_rows_past_4_gib():
    g = _gen(53)
    K, N, T = 4096, 72, 1060001
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, wrapped = i8(T, K), 2 ** 32 // K
    xs = torch.rand(T, device="cuda", generator=g) + 0.1
    for R in (7, 700):
        w, ws = i8(2, N, K), (torch.rand(2, N, device="cuda", generator=g) + 0.1) / K
        rows = torch.randint(wrapped + 1, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        rows[0], rows[-1] = T - 1, wrapped
        first = offsets([R - 3, 3]).cuda()
        at = rows.long()
        ref = ref_int8(x[at], xs[at], w, ws, first, None, R)[0]
        assert_int8(M.grouped_int8_mm(x, xs, w, ws, first, rows=rows, out_dtype=FP32), ref)
        with pytest.raises(AssertionError):           # the bound tells the row 4 GiB before apart
            assert_int8(ref_int8(x[at - wrapped], xs[at], w, ws, first, None, R)[0].float(), ref)


@pytest.mark.parametrize("gathered", [False, True])
def test_weight_gradient_is_held_to_each_groups_own_rows(gathered):
    """Rows outside the groups hold infinities and NaNs; a group's bound counts its own rows."""
    counts, start, tail, N, K = [5, 0, 70, 140, 1], 3, 9, 72, 40
    g = _gen(54)
    R = start + sum(counts) + tail
    first = offsets(counts, start).cuda()
    x, dy = _normal(g, R + 1, K), _normal(g, R, N)
    x[:start], x[R - tail:], dy[:start], dy[R - tail:] = float("nan"), float("inf"), float("inf"), float("nan")
    rows = torch.randint(start, R - tail, (R,), device="cuda", generator=g, dtype=torch.int32) if gathered else None
    if gathered:
        rows[:start] = rows[R - tail:] = R
    dw = M.grouped_mm_dw(dy, x if gathered else x[:R], first, rows=rows)
    ref, mag = ref_dw(dy, x if gathered else x[:R], first, rows)
    for e, c in enumerate(counts):
        assert_product(dw[e], ref[e], mag[e], c)


# ---- grouping

@pytest.mark.parametrize("T,k,E", [(262144, 1, 1024), (262145, 1, 7), (70001, 8, 384), (9001, 64, 1)])
def test_group_routes_of_several_rounds_a_block(T, k, E):
    """At most 262144 routes fit one round of 1024 a block: below, at and past it."""
    g = _gen(T)
    ids = torch.randint(-2, E + 2, (T, k), device="cuda", generator=g, dtype=torch.int32)
    ids[T // 2] = 2 ** 31 - 1
    flat = ids.flatten().long().cpu()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    keys, order = torch.sort(key, stable=True)
    n = int((key < E).sum())
    first, got, token, inverse = (t.cpu() for t in M.group_routes(ids, E))
    assert torch.equal(first.long(), torch.searchsorted(keys, torch.arange(E + 1)))
    assert torch.equal(got[:n].long(), order[:n]) and torch.equal(token[:n].long(), order[:n] // k)
    assert bool((got[n:] == -1).all()) and bool((token[n:] == -1).all())
    want = torch.full((T * k,), -1).scatter(0, order[:n], torch.arange(n))
    assert torch.equal(inverse.flatten().long(), want)
