"""8-bit floating-point products with a scale for each block of 128, their gated block and the quantiser on
the GPU, elementwise against float64 references with derived bounds (tests/gated_util.py)."""
import itertools

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import (FORMS, U, act_bound, assert_close, branches, codes, fp8_bound, ref_act, ref_fp8, ref_quant_fp8)
from products_util import BF16, FP16, FP32, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn

COUNTS = {
    "one": [1],
    "few": [0, 1, 2, 0, 5, 1],
    "mixed": [0, 15, 16, 17, 0, 31, 33, 63, 64, 65, 1, 0],
    "large": [127, 0, 128, 129, 255, 256, 257, 3],
    "many": [(7 * i) % 5 for i in range(200)],
    "empty": [0, 0, 0],
}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _blocks(n):
    return -(-n // 128)


def _scales(g, *shape):
    return torch.empty(*shape, device="cuda").uniform_(0.25, 2.0, generator=g) / 100


def _case(counts, N, K, gathered, glu=False, seed=0):
    """x, x_scales, w, w_scales, first, rows; N outputs (I of a gated block)."""
    g = _gen(seed)
    R, E = sum(counts), len(counts)
    T = max(1, R // 3) if gathered else R
    x, w = codes(g, T, K), codes(g, E, 2 * N if glu else N, K)
    xs = _scales(g, T, _blocks(K))
    ws = _scales(g, E, 2, _blocks(N), _blocks(K)) if glu else _scales(g, E, _blocks(N), _blocks(K))
    ws /= K ** 0.5
    rows = None
    if gathered:
        rows = torch.randint(0, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        if R > 3:
            rows[R // 2], rows[1], rows[-1] = -1, T, 2 ** 31 - 1
    return x, xs, w, ws, offsets(counts).cuda(), rows


def _cut(x, R, w, glu, dtype):
    """Whether a product of these sizes runs the instruction that cuts: 16-bit results in tiles."""
    E, N, K = w.shape
    plan = M.debug_mm_plan(M.MM_FP8_GLU if glu else M.MM_FP8, E, max(R, 1), N // 2 if glu else N, K)
    return dtype != FP32 and plan[0] > 16


def _check(out, case, label="", keep=slice(None)):
    x, xs, w, ws, first, rows = case
    R, K = out.shape[0], x.shape[1]
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, rows, R)
    assert_close(out[keep], ref[keep], fp8_bound(K, mag, top, _cut(x, R, w, False, out.dtype))[keep], label)


def _check_glu(h, case, form, label="", keep=slice(None)):
    x, xs, w, ws, first, rows = case
    R, K = h.shape[0], x.shape[1]
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, rows, R)
    gate, up = branches(ref, form)
    dg, du = branches(fp8_bound(K, mag, top, _cut(x, R, w, True, h.dtype)), form)
    assert_close(h[keep], ref_act(gate, up, form)[keep], act_bound(gate, up, dg, du, form)[keep], label)


# ---- quantiser


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 4112), (70, 256), (5, 7168), (300, 144), (4099, 2064)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantiser(rows, cols, dtype):
    g = _gen(cols)
    x = (torch.randn(rows, cols, device="cuda", generator=g) * torch.rand(rows, 1, device="cuda", generator=g) * 9).to(dtype)
    q, s = M.quant_fp8(x)
    rq, rs = ref_quant_fp8(x)
    assert q.dtype == E4M3 and s.shape == (rows, _blocks(cols))
    assert torch.equal(q.float().double(), rq) and torch.equal(s, rs)


def test_quantiser_on_ties_and_the_ends():
    """Every bf16 and fp16 value against largest magnitudes that put ties on codes' borders; zeros, the smallest
    and largest numbers, infinities and NaN."""
    for dtype in (BF16, FP16):
        every = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(dtype)
        every = every[torch.isfinite(every)]
        for top in (448.0, 1.0, 7.0, 3.5, 0.3, 2.0 ** -14, 2.0 ** -24, 60000.0):
            top = torch.tensor(top, device="cuda").to(dtype)
            v = torch.where(every.abs() <= top, every, 0.0)
            v = torch.nn.functional.pad(v, (0, -len(v) % 127)).view(-1, 127)
            x = torch.cat([v, top.expand(v.shape[0], 1)], 1).contiguous()
            q, s = M.quant_fp8(x)
            rq, rs = ref_quant_fp8(x)
            assert torch.equal(q.float().double(), rq) and torch.equal(s, rs), (dtype, float(top))
    x = torch.zeros(8, 144, dtype=BF16, device="cuda")
    x[1], x[2, 5], x[3, 130], x[4, 0], x[5, 143] = 2.0 ** -133, 3e38, float("inf"), float("nan"), -float("inf")
    x[6, :128], x[7, 3] = torch.linspace(-1, 1, 128, device="cuda") * 2.0 ** -110, -2.0 ** -126
    q, s = M.quant_fp8(x)
    rq, rs = ref_quant_fp8(x)
    assert torch.equal(q.float().double(), rq) and torch.equal(s.isnan(), rs.isnan())
    assert torch.equal(s.nan_to_num(9.0), rs.nan_to_num(9.0))
    assert s.isnan().tolist() == [[False, False]] * 3 + [[False, True], [True, False], [False, True]] + [[False, False]] * 2
    assert s[0].tolist() == [0.0, 0.0] and bool((q[0].float() == 0).all())


def test_quantiser_in_given_buffers_and_past_4_gib():
    rows, cols = 300001, 8192
    x = torch.empty(rows, cols, dtype=BF16, device="cuda").normal_(0, 1, generator=_gen(0))
    q, s = torch.empty(rows, cols, dtype=E4M3, device="cuda"), torch.empty(rows, 64, device="cuda")
    got = M.quant_fp8(x, out=q, scales=s)
    assert got[0] is q and got[1] is s and (q._version, s._version) == (1, 1)
    at = torch.tensor([0, (1 << 31) // cols - 1, (1 << 31) // cols, (1 << 30) // cols, rows - 1], device="cuda")
    rq, rs = ref_quant_fp8(x[at])
    assert torch.equal(q.view(torch.uint8)[at].view(E4M3).float().double(), rq) and torch.equal(s[at], rs)


# ---- products


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K,gathered,out_dtype", [(72, 48, True, BF16), (264, 528, False, FP32), (136, 128, True, FP16),
                                                    (1152, 256, False, BF16), (200, 2064, True, BF16)])
def test_grouped_product(counts, N, K, gathered, out_dtype):
    case = _case(COUNTS[counts], N, K, gathered)
    out = M.grouped_fp8_mm(*case[:5], rows=case[5], out_dtype=out_dtype)
    assert out.dtype == out_dtype and out.shape == (sum(COUNTS[counts]), N)
    _check(out, case)


@pytest.mark.parametrize("M_,N,K", [(1, 8, 16), (1, 4608, 7168), (5, 72, 48), (8, 4608, 1024), (16, 520, 272), (17, 264, 144),
                                    (128, 136, 4096), (500, 392, 528), (2049, 1032, 160), (300, 64, 8192)])
@pytest.mark.parametrize("out_dtype", [None, FP16, FP32])
def test_dense_product(M_, N, K, out_dtype):
    case = _case([M_], N, K, False, seed=K)
    x, xs, w, ws = case[:4]
    out = M.fp8_mm(x, xs, w[0], ws[0], out_dtype=out_dtype)
    assert out.dtype == (out_dtype or BF16)
    _check(out, case)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I,K,gathered,form", [(72, 48, True, "plain"), (264, 528, False, "clamped"), (576, 256, True, "shifted"),
                                               (136, 2064, False, "gate_up")])
def test_grouped_gated_block(counts, I, K, gathered, form):
    case = _case(COUNTS[counts], I, K, gathered, glu=True)
    for dt in (BF16, FP32):
        h = M.grouped_fp8_glu(*case[:5], rows=case[5], out_dtype=dt, **FORMS[form])
        _check_glu(h, case, FORMS[form])


@pytest.mark.parametrize("M_,I,K", [(1, 8, 16), (3, 576, 7168), (17, 264, 144), (500, 392, 528), (300, 64, 8192)])
@pytest.mark.parametrize("form", ["clamped", "situ", "situ_gate_up"])
def test_dense_gated_block(M_, I, K, form):
    case = _case([M_], I, K, False, glu=True, seed=K)
    x, xs, w, ws = case[:4]
    _check_glu(M.fp8_glu(x, xs, w[0], ws[0], out_dtype=FP16, **FORMS[form]), case, FORMS[form])


TILES = [(16, 16), (64, 128), (128, 128), (128, 256), (256, 128)]


def sizes_for(op, shape, parts, reductions=(144, 272, 528, 1040, 2064, 4112)):
    """The least sizes of a list, (counts, N, K), for which the plan names this shape and these parts of the
    reduction (0: of the last round's tiles)."""
    found = None
    for c, e, n, k in itertools.product([11, 70, 130, 260, 600, 1000, 2561], [3, 9, 12, 24, 40],
                                        [72, 136, 264, 520, 600, 1032, 2056], reductions):
        counts = [c + 3, 0, c - 2] + [c] * (e - 3)
        if (found is None or sum(counts) * n * k < found[0]) and M.debug_mm_plan(op, e, sum(counts), n, k) == (*shape, parts):
            found = (sum(counts) * n * k, counts, n, k)
    assert found, f"no sizes with tiles of {shape}"
    return found[1:]


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("shape", TILES)
@pytest.mark.parametrize("glu", [False, True])
def test_tiles(shape, gathered, glu):
    """Every tile shape over two blocks of K and a short one, with NaN codes and scales next to rows and columns
    that are not theirs, and rows outside the groups."""
    counts, N, K = sizes_for(M.MM_FP8_GLU, (shape[0], shape[1] // 2), 1) if glu else sizes_for(M.MM_FP8, shape, 1)
    R = sum(counts)
    x, xs, w, ws, first, rows = _case(counts, N, K, False, glu=glu, seed=N)
    if gathered:
        rows = torch.randperm(R, device="cuda", generator=_gen(3)).to(torch.int32)
    first[-1] -= 1
    call = (lambda o, *a: M.grouped_fp8_glu(*a, first, rows=rows, out=o, limit=2.0)) if glu else (
        lambda o, *a: M.grouped_fp8_mm(*a, first, rows=rows, out=o))
    out = torch.full((R, N), 7.5, dtype=BF16, device="cuda")
    call(out, x, xs, w, ws)
    case = (x, xs, w, ws, first, rows)
    if glu:
        _check_glu(out, case, dict(limit=2.0), keep=slice(0, -1))
    else:
        _check(out, case, keep=slice(0, -1))
    assert bool((out[-1] == 7.5).all())
    bad, f = counts[0] - 1, first.tolist()
    xb, wb, xsb = x.view(torch.uint8).clone(), w.view(torch.uint8).clone(), xs.clone()
    src = int(rows[bad]) if gathered else bad
    src2 = int(rows[bad - 1]) if gathered else bad - 1
    xb[src, K - 1] = 0x7F
    xsb[src2, -1] = float("inf")
    wb[2, 7, 0] = 0xFF
    got = torch.full_like(out, 7.5)
    call(got, xb.view(E4M3), xsb, wb.view(E4M3), ws)
    touched = torch.zeros(R, N, dtype=torch.bool, device="cuda")
    touched[bad] = touched[bad - 1] = True
    touched[f[2]:f[3], 7] = True
    assert torch.equal(got[~touched], out[~touched])
    assert bool(got[bad].isnan().all()) and bool(got[f[2]:f[3], 7].isnan().all())
    assert not bool(torch.isfinite(got[bad - 1]).all())


@pytest.mark.parametrize("out_dtype", [BF16, FP32])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("shape", [(128, 256), (256, 128)])
def test_last_rounds_in_parts(shape, glu, out_dtype):
    """The tiles of a last round, split and joined, with scratch full of NaN; fp32 results take other tiles."""
    op = M.MM_FP8_GLU if glu else M.MM_FP8
    try:
        counts, N, K = sizes_for(op, (shape[0], shape[1] // 2) if glu else shape, 0)
    except AssertionError:
        assert shape == (256, 128)            # (128 x 256 is the better of the two almost everywhere)
        return
    R, E = sum(counts), len(counts)
    x, xs, w, ws, first, rows = _case(counts, N, K, True, glu=glu, seed=N)
    first[-1] -= 2
    scratch = torch.full((M.mm_scratch_bytes(op, E, R, N, K),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((R, N), 7.5, dtype=out_dtype, device="cuda")
    call = M.grouped_fp8_glu if glu else M.grouped_fp8_mm
    call(x, xs, w, ws, first, rows=rows, out=out, scratch=scratch)
    case = (x, xs, w, ws, first, rows)
    if glu:
        _check_glu(out, case, {}, keep=slice(0, -2))
    else:
        _check(out, case, keep=slice(0, -2))
    assert bool((out[-2:] == 7.5).all())
    assert torch.equal(call(x, xs, w, ws, first, rows=rows, out_dtype=out_dtype)[:-2], out[:-2])


@pytest.mark.parametrize("counts,N,K", [([300], 64, 8192), ([90, 0, 140], 72, 8192), ([200], 72, 8208)])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("gathered", [False, True])
def test_split_reductions(counts, N, K, glu, gathered):
    R = sum(counts)
    assert M.debug_mm_plan(M.MM_FP8_GLU if glu else M.MM_FP8, len(counts), R, N, K)[2] > 1
    x, xs, w, ws, first, rows = _case(counts, N, K, gathered, glu=glu)
    first[-1] -= 1
    for dt in (BF16, FP32):
        out = torch.full((R, N), 7.5, dtype=dt, device="cuda")
        (M.grouped_fp8_glu if glu else M.grouped_fp8_mm)(x, xs, w, ws, first, rows=rows, out=out)
        if glu:
            _check_glu(out, (x, xs, w, ws, first, rows), {}, keep=slice(0, -1))
        else:
            _check(out, (x, xs, w, ws, first, rows), keep=slice(0, -1))
        assert bool((out[-1] == 7.5).all())


@pytest.mark.parametrize("glu", [False, True])
def test_last_rounds_of_a_dense_product(glu):
    """More tiles than a round has, the rest in parts."""
    T, N, K = 4097, 2304 if glu else 4608, 4112
    assert M.debug_mm_plan(M.MM_FP8_GLU if glu else M.MM_FP8, 1, T, N, K)[2] == 0
    x, xs, w, ws, first, _ = _case([T], N, K, False, glu=glu, seed=K)
    case = (x, xs, w, ws, first, None)
    if glu:
        _check_glu(M.fp8_glu(x, xs, w[0], ws[0]), case, {})
    else:
        _check(M.fp8_mm(x, xs, w[0], ws[0]), case)


# pairs of scales whose product leaves fp32's range, or whose x scale times the sum does, while the result
# is a number of fp32 (or, at the last, passes it)
ROW_SCALES = [1e-22, 2.4e36, 1.0, 1e-37, 2.0 ** -149, 3e30, -1e-30, 0.0]
COLUMN_SCALES = [1e-22, 200.0, 1e-30, 2.0 ** -149, -1e-3, 3e36, 1.0, 0.0]


@pytest.mark.parametrize("counts,K", [([5], 1040), ([3, 0, 8], 272), ([700, 0, 333], 272), ([90, 0, 140], 8192)])
@pytest.mark.parametrize("out_dtype", [BF16, FP32])
def test_scales_at_the_ends_of_the_range(counts, K, out_dtype):
    """Streamed rows, tiles and split reductions. A row has one scale in all its blocks and a block of columns
    one of its own, so that a result is one product of scales times a sum that rounds as any other; a block's
    sum below 2^-126 may be rounded to a multiple of 2^-149 or to 0 before its factor, below 4: 2^-124 a block.
    Results within a factor of two of the type's largest may be infinite or not."""
    g = _gen(K)
    R, E, N = sum(counts), len(counts), 1032
    x, w = codes(g, R, K), codes(g, E, N, K)
    x.view(torch.uint8)[1::5] = 0
    kb, nb = _blocks(K), _blocks(N)
    xs = torch.tensor(ROW_SCALES, device="cuda").repeat(R // 8 + 1)[:R, None].repeat(1, kb).contiguous()
    ws = torch.tensor(COLUMN_SCALES, device="cuda").repeat(2)[:nb].view(1, nb, 1).repeat(E, 1, kb).contiguous()
    first = offsets(counts).cuda()
    out = M.grouped_fp8_mm(x, xs, w, ws, first, out_dtype=out_dtype).double()
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, None, R)
    fi = torch.finfo(out_dtype)
    bound = fp8_bound(K, mag, top, _cut(x, R, w, False, out_dtype)) + kb * 2.0 ** -124
    tol = bound + (fi.eps / 2) * (ref.abs() + bound) + fi.tiny * fi.eps / 2
    near = mag > fi.max / 2                       # a partial sum may pass the type's range
    ok = ((out - ref).abs() <= tol) | near
    assert bool(ok.all()), ok.logical_not().nonzero()[:5].tolist()
    sure = ref.abs() > fi.max * 2
    assert not bool(torch.isfinite(out[sure]).any())   # (a partial sum may pass the range first, with its own sign)
    assert bool((out[1::5] == 0).all())


def test_rows_of_the_largest_magnitudes():
    """bf16 rows of 3e38: orthogonal ones stay zero with large scales, and small ones bring them into range."""
    x = torch.zeros(2, 256, dtype=BF16, device="cuda")
    x[0, :128], x[1, 128:] = 3e38, 1.0
    q, s = M.quant_fp8(x)
    w = q.repeat(4, 1).contiguous()
    out = M.fp8_mm(q, s, w, torch.full((1, 2), 4e3, device="cuda"), out_dtype=FP32)
    assert out[0, 1::2].tolist() == [0.0] * 4 and out[1, 0::2].tolist() == [0.0] * 4
    assert bool(torch.isinf(out[0, 0::2]).all())
    small = M.fp8_mm(q, s, w, torch.full((1, 2), 1e-30, device="cuda"), out_dtype=FP32)
    want = 448.0 ** 2 * 128 * float(s[0, 0]) * float(torch.tensor(1e-30))
    assert abs(float(small[0, 0]) / want - 1) < 2.0 ** -16


@pytest.mark.parametrize("R,N,K", [(5, 72, 272), (200, 72, 272)])
def test_x_without_rows(R, N, K):
    g = _gen(2)
    x, xs = torch.zeros(0, K, dtype=E4M3, device="cuda"), torch.zeros(0, _blocks(K), device="cuda")
    w, ws = codes(g, 1, N, K), _scales(g, 1, _blocks(N), _blocks(K))
    rows = torch.zeros(R, dtype=torch.int32, device="cuda")
    assert bool((M.grouped_fp8_mm(x, xs, w, ws, offsets([R]).cuda(), rows=rows) == 0).all())
    assert M.fp8_mm(x, xs, w[0], ws[0]).shape == (0, N)


def test_exact_sums():
    """Small whole codes and scales of powers of two: every sum is exact, whatever the order."""
    for M_, N, K in ((5, 264, 4112), (300, 264, 400), (700, 1032, 272)):
        g = _gen(M_)
        ints = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=g).float().to(E4M3)  # noqa: E731
        x, w = ints(M_, K), ints(N, K)
        xs = 2.0 ** torch.randint(-3, 3, (M_, _blocks(K)), device="cuda", generator=g)
        ws = 2.0 ** torch.randint(-3, 3, (_blocks(N), _blocks(K)), device="cuda", generator=g)
        ref = ref_fp8(x, xs, w[None], ws[None], offsets([M_]), None, M_)[0]
        assert torch.equal(M.fp8_mm(x, xs, w, ws, out_dtype=FP32).double(), ref)


def test_gathered_rows_past_4_gib():
    """Rows of x on both sides of 2^31 and 2^32 bytes, streamed and tiled."""
    K, T = 4096, 1100000
    x = torch.zeros(T, K, dtype=torch.uint8, device="cuda")
    g = _gen(5)
    spots = torch.tensor([0, (1 << 31) // K - 1, (1 << 31) // K, (1 << 32) // K - 1, (1 << 32) // K, T - 1], device="cuda")
    x[spots] = codes(g, 6, K).view(torch.uint8)
    xs = torch.zeros(T, 32, device="cuda")
    xs[spots] = _scales(g, 6, 32)
    w, ws = codes(g, 1, 136, K), _scales(g, 1, 2, 32)
    small = x[spots].view(E4M3)
    for R in (6, 600):
        rows = spots[torch.arange(R, device="cuda") % 6].to(torch.int32)
        out = M.grouped_fp8_mm(x.view(E4M3), xs, w, ws, offsets([R]).cuda(), rows=rows)
        _check(out, (small.view(torch.uint8).repeat(R // 6, 1).view(E4M3), xs[spots].repeat(R // 6, 1), w, ws, offsets([R]), None))


@pytest.mark.parametrize("T,N,K", [(3, 1 << 20, 16), (70, 1 << 20, 16), (1, 8, 1 << 20), (37, 16, 1 << 20)])
@pytest.mark.parametrize("out_dtype", [BF16, FP32])
def test_largest_sizes(T, N, K, out_dtype):
    case = _case([T], N, K, False, seed=T)
    x, xs, w, ws = case[:4]
    _check(M.fp8_mm(x, xs, w[0], ws[0], out_dtype=out_dtype), case)
    q, s = M.quant_fp8(torch.randn(2, K, device="cuda", generator=_gen(1)).to(BF16))
    assert q.shape == (2, K) and bool((s > 0).all())


def test_most_groups_most_of_them_empty():
    counts = [0] * 1024
    counts[0], counts[511], counts[1000], counts[1023] = 3, 40, 150, 1
    for glu in (False, True):
        case = _case(counts, 72, 144, True, glu=glu)
        if glu:
            _check_glu(M.grouped_fp8_glu(*case[:5], rows=case[5]), case, {})
        else:
            _check(M.grouped_fp8_mm(*case[:5], rows=case[5]), case)


def test_offsets_that_go_wrong_stay_in_bounds():
    """Offsets beyond R, below 0 or falling cost rows, never a fault; a correct group next to them is right."""
    x, xs, w, ws, _, _ = _case([40, 0, 0], 72, 144, False)
    for f in ([0, 20, 90, 1 << 30], [-5, 20, 10, 40], [0, 20, -(1 << 31), (1 << 31) - 1]):
        first = torch.tensor(f, dtype=torch.int32, device="cuda")
        out = M.grouped_fp8_mm(x, xs, w, ws, first)
        torch.cuda.synchronize()
        if f[2] >= 0:
            _check(out[:10].contiguous(), (x[:10], xs[:10], w[:1], ws[:1], offsets([10]), None))


# ---- the operators together


@pytest.mark.parametrize("T,k,E,K,I", [(8, 6, 64, 528, 144), (300, 2, 6, 272, 144)])
def test_layer_of_fp8_experts(T, k, E, K, I):
    """Routes, quantiser, gated block, quantiser, down product: each stage held to its bound on what the stage
    before it gave; the whole within the formats' precision of the layer in float64."""
    g = _gen(T)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    first, order, token, inverse = M.group_routes(ids, E)
    x = torch.randn(T, K, device="cuda", generator=g).to(BF16)
    w13, w2 = codes(g, E, 2 * I, K), codes(g, E, K, I)
    s13 = _scales(g, E, 2, _blocks(I), _blocks(K)) / K ** 0.5
    s2 = _scales(g, E, _blocks(K), _blocks(I)) / I ** 0.5
    xq, xs = M.quant_fp8(x)
    h = M.grouped_fp8_glu(xq, xs, w13, s13, first, rows=token, limit=7.0)
    hq, hs = M.quant_fp8(h)
    y = M.grouped_fp8_mm(hq, hs, w2, s2, first, out_dtype=FP32)
    R = T * k
    rq, rs = ref_quant_fp8(x)
    assert torch.equal(xq.float().double(), rq) and torch.equal(xs, rs)
    assert h.shape == (R, I)
    _check_glu(h, (xq, xs, w13, s13, first, token), dict(limit=7.0))
    rq, rs = ref_quant_fp8(h)
    assert torch.equal(hq.float().double(), rq) and torch.equal(hs, rs)
    _check(y, (hq, hs, w2, s2, first, None))


def test_captured_layer_replays():
    counts, I, K = [40, 0, 200, 13, 2], 136, 272
    g = _gen(3)
    R, E = sum(counts), len(counts)
    first = offsets(counts).cuda()
    x = torch.randn(R, K, device="cuda", generator=g).to(BF16)
    w13, s13 = codes(g, E, 2 * I, K), _scales(g, E, 2, _blocks(I), _blocks(K)) / 16
    w2, s2 = codes(g, E, 264, 144), _scales(g, E, 3, 2) / 12

    def step():
        h = M.grouped_fp8_glu(*M.quant_fp8(x), w13, s13, first)
        hq, hs = M.quant_fp8(torch.nn.functional.pad(h, (0, 8)))
        return h, hq.view(torch.uint8), hs, M.grouped_fp8_mm(hq, hs, w2, s2, first)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (4, 5, 6):
        x.copy_(torch.randn(R, K, device="cuda", generator=_gen(seed)))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_two_split_calls_at_once_on_two_streams():
    a, b = _case([300], 64, 8192, False, seed=1), _case([300], 64, 8192, False, seed=2)
    assert M.mm_scratch_bytes(M.MM_FP8, 1, 300, 64, 8192) > 0
    want = [M.grouped_fp8_mm(*c[:5]) for c in (a, b)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [M.grouped_fp8_mm(*c[:5], stream=q) for c, q in ((a, s), (b, t))]
        s.synchronize(), t.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
