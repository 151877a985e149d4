"""The gated block's product, its backward pass and the activation's gradient on the GPU, elementwise against
float64 references with derived bounds (tests/gated_util.py)."""
import itertools

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import FORMS, check_backward, check_forward, branches, joined, ref_act, ref_grad
from products_util import BF16, FP16, FP32, assert_product, offsets, ref_dw, ref_dx, ref_mm

pytestmark = pytest.mark.gpu

COUNTS = {
    "one": [1],
    "few": [0, 1, 2, 0, 5, 1],
    "mixed": [0, 15, 16, 17, 0, 31, 33, 63, 64, 65, 1, 0],
    "large": [127, 0, 128, 129, 255, 256, 257, 3],
    "single": [300],
    "many": [(7 * i) % 5 for i in range(200)],
    "empty": [0, 0, 0],
}
SHAPES = [(8, 8), (72, 40), (136, 264), (200, 512), (576, 320)]   # (I, K)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=BF16, scale=1.0):
    return torch.randn(*shape, device="cuda", generator=g).mul_(scale).to(dtype)


def _forward_case(counts, I, K, dtype, gathered, seed=0):
    g = _gen(seed)
    R, E = sum(counts), len(counts)
    T = max(1, R // 3) if gathered else R
    x, w = _normal(g, T, K, dtype=dtype), _normal(g, E, 2 * I, K, dtype=dtype, scale=2 / K ** 0.5)
    rows = None
    if gathered:
        rows = torch.randint(0, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        if R > 3:
            rows[R // 2], rows[1], rows[-1] = -1, T, 2 ** 31 - 1
    return x, w, offsets(counts).cuda(), rows


def _backward_case(counts, N, I, dtype, seed=0, scale=2.0):
    g = _gen(seed)
    R, E = sum(counts), len(counts)
    return (_normal(g, R, N, dtype=dtype), _normal(g, E, N, I, dtype=dtype, scale=1 / N ** 0.5),
            _normal(g, R, 2 * I, dtype=dtype, scale=scale), offsets(counts).cuda())


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I,K", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype,gathered,form", [(BF16, BF16, True, "clamped"), (FP16, FP32, False, "shifted")])
def test_forward(counts, I, K, dtype, out_dtype, gathered, form):
    x, w, first, rows = _forward_case(COUNTS[counts], I, K, dtype, gathered)
    R = sum(COUNTS[counts])
    h, pre = M.grouped_glu(x, w, first, rows=rows, keep_pre=True, out_dtype=out_dtype, **FORMS[form])
    assert h.dtype == out_dtype and pre.dtype == dtype and h.shape == (R, I) and pre.shape == (R, 2 * I)
    ref, mag, _ = ref_mm(x, w, first, rows, R)
    check_forward(h, pre, ref, mag, K, FORMS[form])
    alone = M.grouped_glu(x, w, first, rows=rows, out_dtype=out_dtype, **FORMS[form])
    assert torch.equal(alone, h)


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("I,N", SHAPES)
@pytest.mark.parametrize("dtype,form", [(BF16, "clamped"), (FP16, "shifted")])
def test_backward_through_the_down_product(counts, I, N, dtype, form):
    dy, w, pre, first = _backward_case(COUNTS[counts], N, I, dtype)
    d_pre, h = M.grouped_glu_dx(dy, w, pre, first, keep_h=True, **FORMS[form])
    dh, mag, _ = ref_dx(dy, w, first)
    check_backward(d_pre, h, dh, (N + 1) * 2.0 ** -24 * mag, pre, FORMS[form])
    assert torch.equal(M.grouped_glu_dx(dy, w, pre, first, **FORMS[form]), d_pre)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("R", [3, 150])
def test_forms(form, dtype, R):
    """Streamed and tiled, forward and backward, in each form."""
    I, K = 136, 72
    x, w, first, _ = _forward_case([R], I, K, dtype, False, seed=R)
    h, pre = M.glu(x, w[0], keep_pre=True, out_dtype=FP32, **FORMS[form])
    ref, mag, _ = ref_mm(x, w, first, None, R)
    check_forward(h, pre, ref, mag, K, FORMS[form], "dense")
    gh, gpre = M.grouped_glu(x, w, first, keep_pre=True, out_dtype=FP32, **FORMS[form])
    check_forward(gh, gpre, ref, mag, K, FORMS[form], "grouped")
    dy, wd, pre, first = _backward_case([R], K, I, dtype, seed=R)
    dh, mag, _ = ref_dx(dy, wd, first)
    d_pre, h = M.glu_dx(dy, wd[0], pre, keep_h=True, **FORMS[form])
    check_backward(d_pre, h, dh, (K + 1) * 2.0 ** -24 * mag, pre, FORMS[form], "dense")
    dh = _normal(_gen(R), R, I, dtype=dtype)
    d_pre, h = M.glu_grad(dh, pre, keep_h=True, **FORMS[form])
    check_backward(d_pre, h, dh.double(), 0.0, pre, FORMS[form], "from dh")


@pytest.mark.parametrize("R,I", [(1, 8), (1, 4096), (5, 72), (129, 576), (1000, 1032), (4099, 2048)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_gradient_from_memory(R, I, dtype):
    g = _gen(R)
    dh, pre = _normal(g, R, I, dtype=dtype), _normal(g, R, 2 * I, dtype=dtype, scale=3.0)
    d_pre, h = M.glu_grad(dh, pre, limit=2.5, keep_h=True)
    check_backward(d_pre, h, dh.double(), 0.0, pre, dict(limit=2.5))
    assert torch.equal(M.glu_grad(dh, pre, limit=2.5), d_pre)


@pytest.mark.parametrize("form", ["plain", "clamped", "shifted", "unclamped_alpha"])
def test_gradient_at_the_ends(form):
    """Projections over the whole range: large ones of either sign, zeros of both signs, the limit itself, which
    the gradient passes, and the next values on either side of it."""
    f = FORMS[form]
    L = f.get("limit", 1.5)
    edge = torch.tensor([L, L * (1 + 2 ** -7), L * (1 - 2 ** -8)], dtype=BF16).tolist()
    v = [0.0, -0.0, 1.0, -1.0, 20.0, -20.0, 87.0, -87.0, 90.0, -90.0, 104.0, -104.0, 149.0, -149.0, 300.0, -300.0, 3e4,
         -3e4, 1e-30, -1e-30, 1e18, -1e18] + edge + [-e for e in edge] + [2.0 ** -133]
    v += [0.5] * (-len(v) % 8)
    n = len(v)
    gate, up = torch.tensor(v).repeat_interleave(n), torch.tensor(v).repeat(n)
    gate, up = gate.to(BF16).cuda().view(n, n), up.to(BF16).cuda().view(n, n)
    pre = joined(gate, up, f)
    dh = torch.ones(n, n, dtype=BF16, device="cuda")
    d_pre, h = M.glu_grad(dh, pre, keep_h=True, **f)
    check_backward(d_pre, h, dh.double(), 0.0, pre, f)
    if "limit" in f:
        dg, du = branches(d_pre, f)
        assert bool((dg[gate > L] == 0).all()) and bool((du[up.abs() > L] == 0).all())
        assert bool((du[(up.abs() == L) & (gate == 1)] != 0).all()) and bool((dg[(gate == L) & (up == 1)] != 0).all())


def test_nan_projections_reach_both_gradients():
    """A NaN is not clamped away: h and what depends on it are NaN, the neighbours are not."""
    for f in (FORMS["plain"], FORMS["clamped"], FORMS["situ"]):
        for where in (0, 1):
            gate, up = torch.ones(2, 8, dtype=FP16, device="cuda"), torch.ones(2, 8, dtype=FP16, device="cuda")
            (gate, up)[where][0, 3] = float("nan")
            d_pre, h = M.glu_grad(torch.ones(2, 8, dtype=FP16, device="cuda"), joined(gate, up, f), keep_h=True, **f)
            dg, du = branches(d_pre, f)
            want = torch.zeros(2, 8, dtype=torch.bool, device="cuda")
            want[0, 3] = True
            assert torch.equal(h.isnan(), want)
            assert torch.equal(dg.isnan(), want) and (where == 1 or torch.equal(du.isnan(), want))
    x, w = torch.ones(3, 8, dtype=BF16, device="cuda"), torch.zeros(16, 8, dtype=BF16, device="cuda")
    w[8 + 2, 1] = float("nan")              # gate of column 2
    w[5, 1] = float("nan")                  # up of column 5
    h = M.glu(x, w, limit=1.0)
    assert h.isnan().sum(0).tolist() == [0, 0, 3, 0, 0, 3, 0, 0]


@pytest.mark.parametrize("form", ["plain", "shifted", "situ"])
def test_gradient_matches_differences(form):
    """glu_grad against central differences of glu itself. With an identity for weights the projections are x,
    exactly. The differences of fp32 values at a step of 2^-6 are off by a sixth of its square times the third
    derivative (g sigmoid(g)'s is below 0.6, SiTU's below 2 with the tanh, 1.702^2 for alpha; times up's
    size) and by 2^-18 or so of rounding; the gradient's own rounding in fp16 is 2^-11 of it."""
    f = dict(FORMS[form])
    f.pop("limit", None)
    K = 8
    g = _gen(11)
    x = torch.randint(-96, 97, (64, K), device="cuda", generator=g).to(FP16) / 32    # multiples of 2^-5, exact with the step
    w = torch.cat([torch.eye(K), torch.eye(K).roll(1, 1)]).to(FP16).cuda()          # up = x, gate = x rolled
    h, pre = M.glu(x, w, keep_pre=True, out_dtype=FP32, **f)
    assert torch.equal(pre, torch.cat([x, x.roll(-1, 1)], 1))
    dh = torch.ones(64, K, dtype=FP16, device="cuda")
    d_pre = M.glu_grad(dh, pre, **f).double()
    step = 2.0 ** -6
    for c in range(K):
        up, down = x.clone(), x.clone()
        up[:, c] += step
        down[:, c] -= step
        diff = (M.glu(up, w, out_dtype=FP32, **f).double() - M.glu(down, w, out_dtype=FP32, **f).double()) / (2 * step)
        # x's column c is up of output c and gate of output c - 1
        for got, want in ((d_pre[:, c], diff[:, c]), (d_pre[:, K + (c - 1) % K], diff[:, (c - 1) % K])):
            tol = step ** 2 / 6 * 6.0 * 5.0 + 2.0 ** -16 + 2.0 ** -11 * want.abs()
            assert bool(((got - want).abs() <= tol).all())


@pytest.mark.parametrize("I,K", [(72, 40), (264, 512)])
def test_rows_outside_the_groups_stay(I, K):
    counts, start, tail = [5, 0, 70, 140], 3, 9
    R = start + sum(counts) + tail
    g = _gen(1)
    first = offsets(counts, start).cuda()
    x, w = _normal(g, R, K), _normal(g, 4, 2 * I, K, scale=K ** -0.5)
    x[:start], x[-tail:] = float("nan"), float("inf")
    inside = slice(start, R - tail)
    h, pre = torch.full((R, I), 7.5, dtype=BF16, device="cuda"), torch.full((R, 2 * I), 7.5, dtype=BF16, device="cuda")
    got = M.grouped_glu(x, w, first, out=h, pre=pre, limit=1.0)
    assert got[0] is h and got[1] is pre
    ref, mag, _ = ref_mm(x, w, first, None, R)
    check_forward(h[inside], pre[inside], ref[inside], mag[inside], K, dict(limit=1.0))
    dy, wd = _normal(g, R, K), _normal(g, 4, K, I, scale=K ** -0.5)
    dy[:start], dy[-tail:] = float("inf"), float("nan")
    kept = pre.clone()
    d_pre, h2 = torch.full_like(pre, 7.5), torch.full_like(h, 7.5)
    M.grouped_glu_dx(dy, wd, kept, first, out=d_pre, h=h2, limit=1.0)
    dh, mag, _ = ref_dx(dy, wd, first)
    check_backward(d_pre[inside], h2[inside], dh[inside], (K + 1) * 2.0 ** -24 * mag[inside], kept[inside], dict(limit=1.0))
    for t in (h, pre, d_pre, h2):
        assert bool((t[:start] == 7.5).all()) and bool((t[-tail:] == 7.5).all())


TILES = [(16, 8), (64, 64), (128, 64), (128, 128), (256, 64)]
TILES_DX = [(64, 128), (128, 128), (128, 256), (256, 128)]


def plan_of(op, counts, I, reduction):
    n, k = (reduction, I) if op == M.MM_GLU_DX else (I, reduction)
    return M.debug_mm_plan(op, len(counts), sum(counts), n, k)


def sizes_for(op, shape, parts, reductions=(72, 136, 264, 520, 1032, 2056, 4104)):
    """The least sizes of a list, (counts, I, reduction), for which the plan names this shape and these parts of
    the reduction (0: of the last round's tiles)."""
    found = None
    for c, e, I, k in itertools.product([11, 70, 130, 260, 600, 1000, 2561], [3, 9, 12, 24, 40],
                                        [72, 136, 264, 520, 600, 1032, 2056], reductions):
        counts = [c + 3, 0, c - 2] + [c] * (e - 3)
        if (found is None or sum(counts) * I * k < found[0]) and plan_of(op, counts, I, k) == (*shape, parts):
            found = (sum(counts) * I * k, counts, I, k)
    assert found, f"no sizes with tiles of {shape}"
    return found[1:]


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", TILES)
def test_forward_tiles(shape, dtype, gathered):
    """Infinities and NaNs stay in the rows and columns they belong to, over tiles' ends and groups'."""
    counts, I, K = sizes_for(M.MM_GLU, shape, 1)
    R, E = sum(counts), len(counts)
    g = _gen(I)
    x, w = _normal(g, R, K, dtype=dtype), _normal(g, E, 2 * I, K, dtype=dtype, scale=K ** -0.5)
    rows = torch.randperm(R, device="cuda", generator=g).to(torch.int32) if gathered else None
    first = offsets(counts).cuda()
    h, pre = M.grouped_glu(x, w, first, rows=rows, keep_pre=True)
    ref, mag, _ = ref_mm(x, w, first, rows, R)
    check_forward(h, pre, ref, mag, K, {})
    clean = h
    bad_row, bad_e, bad_c = counts[0] - 1, 2, I + 7
    xb, wb = x.clone(), w.clone()
    xb[rows[bad_row] if gathered else bad_row, K - 1] = float("nan")
    wb[bad_e, bad_c, 0] = float("inf")
    h, pre = M.grouped_glu(xb, wb, first, rows=rows, keep_pre=True)
    f = first.tolist()
    touched = torch.zeros(R, I, dtype=torch.bool, device="cuda")
    touched[bad_row] = True
    touched[f[bad_e]:f[bad_e + 1], 7] = True
    assert torch.equal(h[~touched], clean[~touched])
    assert not bool(torch.isfinite(pre[bad_row]).any()) and not bool(torch.isfinite(pre[f[bad_e]:f[bad_e + 1], bad_c]).any())


TILES_DX = {(64, 128): ([70] * 12, 1200, 72), (128, 128): ([130] * 40, 1032, 72), (128, 256): ([1000] * 9, 2056, 136),
            (256, 128): ([2560] * 6, 2056, 72)}


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", TILES_DX)
def test_backward_tiles(shape, dtype):
    counts, I, N = sizes_for(M.MM_GLU_DX, shape, 1)
    dy, w, pre, first = _backward_case(counts, N, I, dtype, seed=I)
    d_pre, h = M.grouped_glu_dx(dy, w, pre, first, keep_h=True, limit=2.0)
    dh, mag, _ = ref_dx(dy, w, first)
    check_backward(d_pre, h, dh, (N + 1) * 2.0 ** -24 * mag, pre, dict(limit=2.0))
    bad = counts[0] - 1
    dyb, preb = dy.clone(), pre.clone()
    dyb[bad, N - 1], preb[bad + 1, 5] = float("nan"), float("nan")   # (an up branch: its own gradient is gate's)
    d2, h2 = M.grouped_glu_dx(dyb, w, preb, first, keep_h=True, limit=2.0)
    keep = torch.ones_like(d_pre, dtype=torch.bool)
    keep[bad] = False
    keep[bad + 1, 5] = keep[bad + 1, I + 5] = False
    assert torch.equal(d2[keep], d_pre[keep])
    keep_h = torch.ones_like(h, dtype=torch.bool)
    keep_h[bad + 1, 5] = False
    assert torch.equal(h2[keep_h], h[keep_h]) and bool(h2[bad + 1, 5].isnan())
    assert bool(d2[bad + 1, I + 5].isnan()) == (float(pre[bad + 1, I + 5]) <= 2.0)   # (a gate beyond the limit has no gradient)


LAST_ROUNDS = [(M.MM_GLU, (128, 128)), (M.MM_GLU, (256, 64)), (M.MM_GLU_DX, (128, 256)), (M.MM_GLU_DX, (256, 128))]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("op,shape", LAST_ROUNDS)
def test_last_rounds_in_parts(op, shape, dtype):
    """The tiles of a last round, split and joined: every row against the reference, twice the same bits, rows in
    no group left alone, and no tile joined from another call's sums (scratch full of NaN)."""
    counts, I, K = sizes_for(op, shape, 0)
    R, E = sum(counts), len(counts)
    scratch = torch.full((M.mm_scratch_bytes(op, E, R, *((K, I) if op == M.MM_GLU_DX else (I, K))),), 255, dtype=torch.uint8, device="cuda")
    out2, h2 = torch.full((R, 2 * I), 7.5, dtype=dtype, device="cuda"), torch.full((R, I), 7.5, dtype=dtype, device="cuda")
    if op == M.MM_GLU:
        x, w, first, rows = _forward_case(counts, I, K, dtype, True, seed=I)
        first[-1] -= 2
        M.grouped_glu(x, w, first, rows=rows, out=h2, pre=out2, scratch=scratch, limit=1.5)
        ref, mag, _ = ref_mm(x, w, first, rows, R)
        check_forward(h2[:-2], out2[:-2], ref[:-2], mag[:-2], K, dict(limit=1.5))
        h, out = M.grouped_glu(x, w, first, rows=rows, keep_pre=True, limit=1.5)
    else:
        dy, w, pre, first = _backward_case(counts, K, I, dtype, seed=I)
        first[-1] -= 2
        M.grouped_glu_dx(dy, w, pre, first, out=out2, h=h2, scratch=scratch, limit=1.5)
        dh, mag, _ = ref_dx(dy, w, first)
        check_backward(out2[:-2], h2[:-2], dh[:-2], (K + 1) * 2.0 ** -24 * mag[:-2], pre[:-2], dict(limit=1.5))
        out, h = M.grouped_glu_dx(dy, w, pre, first, keep_h=True, limit=1.5)
    assert torch.equal(out[:-2], out2[:-2]) and torch.equal(h[:-2], h2[:-2])
    assert bool((out2[-2:] == 7.5).all()) and bool((h2[-2:] == 7.5).all())


def test_last_rounds_of_a_dense_block():
    """4097 rows: a whole round and a few tiles; and groups so unequal that the estimate of the tiles is far off."""
    g = _gen(4)
    T, I, K = 4097, 2304, 2056
    assert plan_of(M.MM_GLU, [T], I, K)[2] == 0
    x, w = _normal(g, T, K), _normal(g, 2 * I, K, scale=K ** -0.5)
    h, pre = M.glu(x, w, keep_pre=True)
    ref, mag, _ = ref_mm(x, w[None], offsets([T]), None, T)
    check_forward(h, pre, ref, mag, K, {})
    for counts in ([T - 5, 1, 1, 1, 1, 1], [1] * 5 + [T - 5], [700, 0, 700, 0, 2697, 0]):
        w6 = _normal(g, 6, 2 * I, K, scale=K ** -0.5)
        first = offsets(counts).cuda()
        h = M.grouped_glu(x, w6, first)
        ref, mag, _ = ref_mm(x, w6, first, None, T)
        check_forward(h, None, ref, mag, K, {})


@pytest.mark.parametrize("counts,I,K", [([300], 64, 8192), ([90, 0, 140], 72, 8192), ([200], 72, 4096)])
@pytest.mark.parametrize("gathered", [False, True])
def test_split_reductions(counts, I, K, gathered):
    R, E = sum(counts), len(counts)
    assert M.debug_mm_plan(M.MM_GLU, E, R, I, K)[2] > 1 and M.debug_mm_plan(M.MM_GLU_DX, E, R, K, I)[2] > 1
    x, w, first, rows = _forward_case(counts, I, K, BF16, gathered)
    first[-1] -= 1                           # the last row belongs to no group
    h, pre = torch.full((R, I), 7.5, dtype=BF16, device="cuda"), torch.full((R, 2 * I), 7.5, dtype=BF16, device="cuda")
    M.grouped_glu(x, w, first, rows=rows, out=h, pre=pre, **FORMS["clamped"])
    ref, mag, _ = ref_mm(x, w, first, rows, R)
    check_forward(h[:-1], pre[:-1], ref[:-1], mag[:-1], K, FORMS["clamped"])
    dy, wd, pre2, _ = _backward_case(counts, K, I, FP16)
    d_pre, h2 = torch.full((R, 2 * I), 7.5, dtype=FP16, device="cuda"), torch.full((R, I), 7.5, dtype=FP16, device="cuda")
    M.grouped_glu_dx(dy, wd, pre2, first, out=d_pre, h=h2)
    dh, mag, _ = ref_dx(dy, wd, first)
    check_backward(d_pre[:-1], h2[:-1], dh[:-1], (K + 1) * 2.0 ** -24 * mag[:-1], pre2[:-1], {})
    for t in (h, pre, d_pre, h2):
        assert bool((t[-1] == 7.5).all())


@pytest.mark.parametrize("R,I,K", [(5, 72, 272), (200, 72, 272), (200, 136, 40)])
def test_x_without_rows(R, I, K):
    """Every product row is a row of zeros: act(0, 0), and with gate 0 no gate gradient of beta."""
    x = torch.zeros(0, K, dtype=BF16, device="cuda")
    w = _normal(_gen(2), 1, 2 * I, K)
    rows = torch.zeros(R, dtype=torch.int32, device="cuda")
    h, pre = M.grouped_glu(x, w, offsets([R]).cuda(), rows=rows, keep_pre=True, alpha=1.5, beta=2.0)
    assert bool((h == 0).all()) and bool((pre == 0).all())


def test_no_rows_and_no_groups():
    x, w = torch.zeros(0, 16, dtype=BF16, device="cuda"), torch.zeros(2, 16, 16, dtype=BF16, device="cuda")
    first = torch.zeros(3, dtype=torch.int32, device="cuda")
    h, pre = M.grouped_glu(x, w, first, keep_pre=True)
    assert h.shape == (0, 8) and pre.shape == (0, 16)
    assert M.glu(x, w[0]).shape == (0, 8)
    assert M.grouped_glu_dx(torch.zeros(0, 16, dtype=BF16, device="cuda"), torch.zeros(2, 16, 8, dtype=BF16, device="cuda"),
                            pre, first).shape == (0, 16)
    assert M.glu_grad(h, pre).shape == (0, 16)


def test_offsets_that_go_wrong_stay_in_bounds():
    """Offsets beyond R, below 0 or falling cost rows, never a fault; correct groups next to them are right."""
    g = _gen(8)
    x, w = _normal(g, 40, 72), _normal(g, 3, 144, 72, scale=0.2)
    dy, wd, pre = _normal(g, 40, 72), _normal(g, 3, 72, 72, scale=0.2), _normal(g, 40, 144)
    for f in ([0, 20, 90, 1 << 30], [-5, 20, 10, 40], [0, 20, -(1 << 31), (1 << 31) - 1]):
        first = torch.tensor(f, dtype=torch.int32, device="cuda")
        h = M.grouped_glu(x, w, first)
        if f[2] < 0:
            M.grouped_glu_dx(dy, wd, pre, first)
            torch.cuda.synchronize()
            continue                         # the last group takes all rows again
        ref, mag, _ = ref_mm(x[:20], w[:1], offsets([20]), None, 20)
        check_forward(h[:10], None, ref[:10], mag[:10], 72, {})
        d_pre = M.grouped_glu_dx(dy, wd, pre, first)
        dh, mag, _ = ref_dx(dy[:20], wd[:1], offsets([20]))
        check_backward(d_pre[:10], None, dh[:10], 73 * 2.0 ** -24 * mag[:10], pre[:10], {})


def test_last_rounds_of_a_dense_backward():
    """More tiles than a round has, the rest in parts: the estimate is exact for one group."""
    T, I, N = 4097, 4360, 1032
    assert plan_of(M.MM_GLU_DX, [T], I, N)[2] == 0 and T // 128 * (I // 256) >= 512
    dy, w, pre, first = _backward_case([T], N, I, BF16, seed=2)
    d_pre, h = M.glu_dx(dy, w[0], pre, keep_h=True, limit=2.0)
    dh, mag, _ = ref_dx(dy, w, first)
    check_backward(d_pre, h, dh, (N + 1) * 2.0 ** -24 * mag, pre, dict(limit=2.0))


class _GatedExperts(torch.autograd.Function):
    """A routed layer's expert block as a training program wraps it: x [T, K] to the sorted rows' outputs."""

    @staticmethod
    def forward(ctx, x, w13, w2, first, token, inverse, limit):
        h, pre = M.grouped_glu(x, w13, first, rows=token, keep_pre=True, limit=limit)
        ctx.save_for_backward(x, w13, w2, first, token, inverse, pre)
        ctx.limit = limit
        return M.grouped_mm(h, w2, first)

    @staticmethod
    def backward(ctx, dy):
        x, w13, w2, first, token, inverse, pre = ctx.saved_tensors
        d_pre, h = M.grouped_glu_dx(dy.contiguous(), w2, pre, first, keep_h=True, limit=ctx.limit)
        dw2 = M.grouped_mm_dw(dy.contiguous(), h, first)
        dw13 = M.grouped_mm_dw(d_pre, x, first, rows=token)
        dxr = M.grouped_mm_dx(d_pre, w13, first, out_dtype=FP32)
        return dxr[inverse.long()].sum(1).to(x.dtype), dw13, dw2, None, None, None, None


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_training_step_of_a_routed_layer(dtype):
    """Routes, gated block, down product and all gradients in one step, each stage held to its bound on what the
    stage before it gave, and autograd's gradients to those of the calls themselves."""
    T, k, E, K, I, L = 300, 2, 6, 264, 136, 2.0
    g = _gen(21)
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    first, order, token, inverse = M.group_routes(ids, E)
    x = _normal(g, T, K, dtype=dtype).requires_grad_()
    w13 = _normal(g, E, 2 * I, K, dtype=dtype, scale=2 * K ** -0.5).requires_grad_()
    w2 = _normal(g, E, K, I, dtype=dtype, scale=I ** -0.5).requires_grad_()
    y = _GatedExperts.apply(x, w13, w2, first, token, inverse, L)
    dy = _normal(g, T * k, K, dtype=dtype)
    y.backward(dy)
    with torch.no_grad():
        h, pre = M.grouped_glu(x, w13, first, rows=token, keep_pre=True, limit=L)
        ref, mag, cov = ref_mm(x, w13, first, token, T * k)
        assert bool(cov.all())
        check_forward(h, pre, ref, mag, K, dict(limit=L))
        ref, mag, _ = ref_mm(h, w2, first, None, T * k)
        assert_product(y.detach(), ref, mag, I)
        d_pre, h2 = M.grouped_glu_dx(dy, w2, pre, first, keep_h=True, limit=L)
        dh, mag, _ = ref_dx(dy, w2, first)
        check_backward(d_pre, h2, dh, (K + 1) * 2.0 ** -24 * mag, pre, dict(limit=L))
        ref, mag = ref_dw(dy, h2, first, None)
        assert_product(w2.grad, ref, mag, T * k)
        ref, mag = ref_dw(d_pre, x, first, token)
        assert_product(w13.grad, ref, mag, T * k)
        dxr = M.grouped_mm_dx(d_pre, w13, first, out_dtype=FP32)
        assert torch.equal(x.grad, dxr[inverse.long()].sum(1).to(dtype))


def test_captured_step_replays():
    """The block's calls in a graph, replayed on new inputs between eager work on the same scratch-free calls."""
    counts, I, K = [40, 0, 200, 13], 136, 264
    R, E = sum(counts), len(counts)
    g = _gen(3)
    first = offsets(counts).cuda()
    x, w, wd = _normal(g, R, K), _normal(g, E, 2 * I, K, scale=0.1), _normal(g, E, K, I, scale=0.1)
    dy, dh = _normal(g, R, K), _normal(g, R, I)

    def step():
        h, pre = M.grouped_glu(x, w, first, keep_pre=True, limit=1.5)
        d_pre, h2 = M.grouped_glu_dx(dy, wd, pre, first, keep_h=True, limit=1.5)
        return h, pre, d_pre, h2, M.glu_grad(dh, pre, limit=1.5), M.glu(x, w[0])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (4, 5, 6):
        x.copy_(_normal(_gen(seed), R, K))
        dy.copy_(_normal(_gen(seed + 10), R, K))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_two_split_calls_at_once_on_two_streams():
    I, K, R = 72, 8192, 300
    a, b = _forward_case([R], I, K, BF16, False, seed=1), _forward_case([R], I, K, BF16, False, seed=2)
    assert M.mm_scratch_bytes(M.MM_GLU, 1, R, I, K) > 0
    want = [M.grouped_glu(c[0], c[1], c[2]) for c in (a, b)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        got = [M.grouped_glu(c[0], c[1], c[2], stream=q) for c, q in ((a, s), (b, t))]
        s.synchronize(), t.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_given_outputs_advance_their_version_and_keep_autograd_honest():
    x, w = torch.ones(4, 16, dtype=BF16, device="cuda"), torch.ones(16, 16, dtype=BF16, device="cuda")
    h, pre = torch.zeros(4, 8, dtype=BF16, device="cuda"), torch.zeros(4, 16, dtype=BF16, device="cuda")
    M.glu(x, w, out=h, pre=pre)
    assert (h._version, pre._version) == (1, 1)
    out, h2 = torch.zeros(4, 16, dtype=BF16, device="cuda"), torch.zeros(4, 8, dtype=BF16, device="cuda")
    M.glu_grad(h, pre, out=out, h=h2)
    assert (out._version, h2._version, h._version, pre._version) == (1, 1, 1, 1)


def test_gradient_past_4_gib():
    """Projections of 2^33 bytes and more: rows on both sides of 2^31 and 2^32 elements are right."""
    I, R = 4096, 540000
    pre = torch.empty(R, 2 * I, dtype=BF16, device="cuda").normal_(0, 2, generator=_gen(1))
    dh = torch.empty(R, I, dtype=BF16, device="cuda").normal_(0, 1, generator=_gen(2))
    d_pre, h = M.glu_grad(dh, pre, keep_h=True, limit=3.0)
    at = torch.tensor([0, (1 << 31) // (2 * I) - 1, (1 << 31) // (2 * I), (1 << 32) // (2 * I) - 1, (1 << 32) // (2 * I),
                       (1 << 31) // I, R - 1], device="cuda")
    check_backward(d_pre[at], h[at], dh[at].double(), 0.0, pre[at], dict(limit=3.0))


def test_forward_rows_past_4_gib():
    """h and pre past 2^32 bytes, x gathered from two rows."""
    I, K, R = 4096, 16, 300001
    x, w = _normal(_gen(1), 2, K), _normal(_gen(2), 1, 2 * I, K, scale=0.5)
    rows = (torch.arange(R, device="cuda") % 2).to(torch.int32)
    h, pre = M.grouped_glu(x, w, offsets([R]).cuda(), rows=rows, keep_pre=True)
    small, spre = M.grouped_glu(x, w, offsets([2]).cuda(), keep_pre=True)
    ref, mag, _ = ref_mm(x, w, offsets([2]), None, 2)
    check_forward(small, spre, ref, mag, K, {})
    for lo in range(0, R, 50000):
        hi = min(R, lo + 50000)
        check = rows[lo:hi].long()
        assert torch.equal(h[lo:hi], h[:2][check]) and torch.equal(pre[lo:hi], pre[:2][check])
    check_forward(h[:2], pre[:2], ref, mag, K, {})


@pytest.mark.parametrize("R", [6, 603])
def test_gathered_rows_past_4_gib(R):
    """Rows of x on both sides of 2^31 and 2^32 bytes, streamed and tiled; names of no row past them are zeros."""
    K, T, I = 2048, 1100000, 136
    g = _gen(5)
    x = torch.zeros(T, K, dtype=BF16, device="cuda")
    spots = torch.tensor([0, (1 << 31) // (2 * K) - 1, (1 << 31) // (2 * K), (1 << 32) // (2 * K) - 1, (1 << 32) // (2 * K), T - 1],
                         device="cuda")
    x[spots] = _normal(g, 6, K)
    w = _normal(g, 1, 2 * I, K, scale=K ** -0.5)
    rows = spots[torch.arange(R, device="cuda") % 6].to(torch.int32)
    rows[2] = T
    h, pre = M.grouped_glu(x, w, offsets([R]).cuda(), rows=rows, keep_pre=True)
    small = x[spots][torch.arange(R, device="cuda") % 6]
    small[2] = 0
    ref, mag, _ = ref_mm(small, w, offsets([R]), None, R)
    check_forward(h, pre, ref, mag, K, {})


@pytest.mark.parametrize("T,I,K", [(3, 1 << 19, 8), (70, 1 << 19, 8), (1, 8, 1 << 20), (37, 16, 1 << 20)])
def test_largest_sizes(T, I, K):
    """The longest rows and the most columns that a call takes, forward and backward."""
    g = _gen(T)
    x, w = _normal(g, T, K), _normal(g, 2 * I, K, scale=K ** -0.5)
    h, pre = M.glu(x, w, keep_pre=True, limit=2.0)
    ref, mag, _ = ref_mm(x, w[None], offsets([T]), None, T)
    check_forward(h, pre, ref, mag, K, dict(limit=2.0))
    dy, wd = _normal(g, T, K), _normal(g, K, I, scale=K ** -0.5)
    d_pre = M.glu_dx(dy, wd, pre, limit=2.0)
    dh, mag, _ = ref_dx(dy, wd[None], offsets([T]))
    check_backward(d_pre, None, dh, (K + 1) * 2.0 ** -24 * mag, pre, dict(limit=2.0))


def test_most_groups_most_of_them_empty():
    counts = [0] * 1024
    counts[0], counts[511], counts[1000], counts[1023] = 3, 40, 150, 1
    x, w, first, rows = _forward_case(counts, 72, 136, FP16, True)
    R = sum(counts)
    h, pre = M.grouped_glu(x, w, first, rows=rows, keep_pre=True)
    ref, mag, _ = ref_mm(x, w, first, rows, R)
    check_forward(h, pre, ref, mag, 136, {})
    dy, wd, pre, first = _backward_case(counts, 136, 72, FP16)
    d_pre, h = M.grouped_glu_dx(dy, wd, pre, first, keep_h=True)
    dh, mag, _ = ref_dx(dy, wd, first)
    check_backward(d_pre, h, dh, 137 * 2.0 ** -24 * mag, pre, {})


def test_two_captured_steps_replayed_at_once():
    """Two graphs, each with split products and last rounds in parts, on two streams: their scratch is their own."""
    cases = [_forward_case([300], 72, 8192, BF16, False, seed=s) for s in (1, 2)]
    backs = [_backward_case([430] + [0] * 3, 4104, 1032, BF16, seed=s) for s in (3, 4)]
    assert plan_of(M.MM_GLU, [300], 72, 8192)[2] > 1

    def step(i):
        x, w, first, _ = cases[i]
        dy, wd, pre, bfirst = backs[i]
        return M.grouped_glu(x, w, first), M.grouped_glu_dx(dy, wd, pre, bfirst)

    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in (0, 1):
        step(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(step(i))
    want = [[t.clone() for t in step(i)] for i in (0, 1)]
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        torch.cuda.synchronize()
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, v))


@pytest.mark.parametrize("R", [5, 300, 2000])
def test_c_abi_gathers_rows_of_one_group(R):
    """Without offsets but with row numbers: one group whose rows of x are named, 16 bits and 8."""
    from block_scaled_fp4_histogram_amd import _lib
    from gated_util import act_bound, assert_close, codes, fp8_bound, ref_fp8
    L, g = _lib.load(), _gen(R)
    T, I, K = 50, 136, 272
    x, w = _normal(g, T, K), _normal(g, 1, 2 * I, K, scale=K ** -0.5)
    rows = torch.randint(-2, T + 2, (R,), device="cuda", generator=g, dtype=torch.int32)
    h, pre = torch.empty(R, I, dtype=BF16, device="cuda"), torch.empty(R, 2 * I, dtype=BF16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    scratch = torch.empty(max(1, M.mm_scratch_bytes(M.MM_GLU, 1, R, I, K)), dtype=torch.uint8, device="cuda")
    assert L.moe_grouped_glu(M.T_BF16, x.data_ptr(), T, rows.data_ptr(), w.data_ptr(), None, 1, R, I, K, None, M.T_BF16,
                             h.data_ptr(), pre.data_ptr(), scratch.data_ptr(), scratch.numel(), stream) == M.MOE_OK
    ref, mag, _ = ref_mm(x, w, offsets([R]), rows, R)
    check_forward(h, pre, ref, mag, K, {})
    xq, wq = codes(g, T, K), codes(g, 1, 2 * I, K)
    xs, ws = torch.rand(T, 3, device="cuda", generator=g) / 100, torch.rand(1, 2, 2, 3, device="cuda", generator=g) / 2000
    scratch = torch.empty(max(1, M.mm_scratch_bytes(M.MM_FP8_GLU, 1, R, I, K)), dtype=torch.uint8, device="cuda")
    out = torch.empty(R, I, dtype=FP32, device="cuda")
    assert L.moe_grouped_fp8_glu(xq.data_ptr(), xs.data_ptr(), T, rows.data_ptr(), wq.data_ptr(), ws.data_ptr(), None, 1, R, I, K,
                                 None, M.T_FP32, out.data_ptr(), scratch.data_ptr(), scratch.numel(), stream) == M.MOE_OK
    ref, mag, top, _ = ref_fp8(xq, xs, wq, ws, offsets([R]), rows, R)
    gate, up = branches(ref, {})
    dg, du = branches(fp8_bound(K, mag, top, False), {})
    assert_close(out, ref_act(gate, up, {}), act_bound(gate, up, dg, du, {}))


@pytest.mark.parametrize("form", ["plain", "shifted", "situ"])
def test_references_agree_with_autograd(form):
    """The formula's gradient that the kernels are held to is autograd's of the definition."""
    f = FORMS[form]
    g = _gen(9)
    pre = torch.randn(40, 48, dtype=torch.float64, device="cuda", generator=g).mul_(2).requires_grad_()
    gate, up = branches(pre, f)
    dh = torch.randn(40, 24, dtype=torch.float64, device="cuda", generator=g)
    ref_act(gate, up, f).backward(dh)
    rg, ru = ref_grad(dh, gate.detach(), up.detach(), f)
    torch.testing.assert_close(pre.grad, joined(rg, ru, f), rtol=1e-12, atol=1e-12)
