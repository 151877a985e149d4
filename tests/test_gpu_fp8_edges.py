"""8-bit floating-point products: that the tiles of a last round are split where the plan says so, for each type of
result, and sums that a cut or a lost term would change, on the GPU."""
import itertools

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import act_bound, assert_close, branches, codes, fp8_bound, ref_act, ref_fp8
from last_round_util import last_round
from products_util import BF16, FP16, FP32, offsets
from test_gpu_fp8 import TILES, sizes_for

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn

FAST_TILES = [(64, 128), (128, 128), (128, 256), (256, 128)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _blocks(n):
    return -(-n // 128)


def _operands(counts, N, K, glu, seed=0):
    g = _gen(seed)
    R, E = sum(counts), len(counts)
    x, w = codes(g, R, K), codes(g, E, 2 * N if glu else N, K)
    xs = torch.empty(R, _blocks(K), device="cuda").uniform_(0.25, 2.0, generator=g) / 100
    ws = torch.empty(*((E, 2) if glu else (E,)), _blocks(N), _blocks(K), device="cuda").uniform_(0.25, 2.0, generator=g)
    return x, xs, w, ws / (100 * K ** 0.5), offsets(counts).cuda()


def split_sizes(glu, groups, op=None, shape=None):
    """The least (counts, N, K) of a list that the plan takes in parts (0), in tiles of `shape` where it is given,
    and whose offsets make a last round that is split."""
    op = op or (M.MM_FP8_GLU if glu else M.MM_FP8)
    found = None
    for c, e, n, k in itertools.product([600, 1000, 1100, 2100, 2561, 4097], groups, [520, 1032, 2056, 2304, 4608], [2064, 4112, 7168]):
        counts = [c] if e == 1 else [c + 3, 0, c - 2] + [c] * (e - 3)
        if found is not None and sum(counts) * n * k >= found[0]:
            continue
        rows, cols, parts = M.debug_mm_plan(op, e, sum(counts), n, k)
        if shape and (rows, cols * (2 if glu else 1)) != shape:
            continue
        if parts == 0 and last_round(counts, n, rows, cols, -(-k // 128))[0] >= 2:
            found = (sum(counts) * n * k, counts, n, k)
    assert found, "no such sizes"
    return found[1:]


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("groups,shape", [([1], None), ([5, 9, 12, 24, 40], (128, 256)), ([5, 9, 12, 24, 40], (256, 128))])
@pytest.mark.parametrize("glu", [False, True])
def test_last_rounds_are_split_and_joined(glu, groups, shape, out_dtype):
    """The plan's 0 parts, the tile count that the offsets make, and the sums that scratch (all ones before) holds
    afterwards agree, so the split and the join have run; and the results are right."""
    counts, N, K = split_sizes(glu, groups, shape=shape)
    op, R, E = M.MM_FP8_GLU if glu else M.MM_FP8, sum(counts), len(counts)
    rows, cols, parts = M.debug_mm_plan(op, E, R, N, K)
    assert parts == 0
    split, words = last_round(counts, N, rows, cols, -(-K // 128), 2 if glu else 1)
    assert split >= 2
    x, xs, w, ws, first = _operands(counts, N, K, glu, seed=K)
    scratch = torch.full((M.mm_scratch_bytes(op, E, R, N, K),), 255, dtype=torch.uint8, device="cuda")
    call = M.grouped_fp8_glu if glu else M.grouped_fp8_mm
    out = call(x, xs, w, ws, first, out_dtype=out_dtype, scratch=scratch)
    assert int((scratch.view(torch.int32) != -1).sum()) == words
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, None, R)
    bound = fp8_bound(K, mag, top, False)
    if glu:
        (gate, up), (dg, du) = branches(ref, {}), branches(bound, {})
        assert_close(out, ref_act(gate, up, {}), act_bound(gate, up, dg, du, {}))
    else:
        assert_close(out, ref, bound)


def _cancelling(counts, N, K, glu, seed):
    """Codes whose every eight products hold 448 x 448 and its negative beside products of small whole numbers, all
    scales 1: any order of fp32 sums is exact (below 2^24), and the results are whole numbers of at most 256, which
    16 bits hold."""
    g = _gen(seed)
    R, E, W = sum(counts), len(counts), 2 * N if glu else N
    ints = lambda top, *s: torch.randint(-top, top + 1, s, device="cuda", generator=g).float()  # noqa: E731
    x = ints(1, R, K) * (torch.rand(R, K, device="cuda", generator=g) < min(1.0, 300 / K))
    w = ints(2, E, W, K)
    x[:, 0::8], x[:, 3::8], w[..., 0::8], w[..., 3::8] = 448.0, -448.0, 448.0, 448.0
    xs = torch.ones(R, _blocks(K), device="cuda")
    ws = torch.ones(*((E, 2) if glu else (E,)), _blocks(N), _blocks(K), device="cuda")
    return x.to(E4M3), xs, w.to(E4M3), ws, offsets(counts).cuda()


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("how", ["streamed", "split", "last round", *TILES[1:]], ids=str)
def test_sums_whose_large_products_cancel(how, glu, out_dtype):
    """Streamed rows, split reductions, last rounds in parts and every tile shape, for each type of result."""
    op = M.MM_FP8_GLU if glu else M.MM_FP8
    if how == "streamed":
        counts, N, K = [5, 0, 9], 264, 528
    elif how == "split":
        counts, N, K = [90, 0, 140], 72, 8192
    elif how == "last round":
        counts, N, K = split_sizes(glu, [1, 5, 9, 12, 24])
    else:
        counts, N, K = sizes_for(op, (how[0], how[1] // 2) if glu else how, 1)
    plan = M.debug_mm_plan(op, len(counts), sum(counts), N, K)
    assert plan[0] == 16 if how == "streamed" else plan[2] > 1 if how == "split" else plan[0] > 16
    x, xs, w, ws, first = _cancelling(counts, N, K, glu, seed=K)
    ref, _, _, _ = ref_fp8(x, xs, w, ws, first, None, sum(counts))
    assert float(ref.abs().max()) <= 256 and float(ref.abs().max()) >= 8
    if glu:
        h = M.grouped_fp8_glu(x, xs, w, ws, first, out_dtype=out_dtype)
        gate, up = branches(ref, {})
        zero = torch.zeros_like(gate)
        assert_close(h, ref_act(gate, up, {}), act_bound(gate, up, zero, zero, {}))
    else:
        assert torch.equal(M.grouped_fp8_mm(x, xs, w, ws, first, out_dtype=out_dtype).double(), ref)


# ---- fast_sums


@pytest.mark.parametrize("out_dtype", [BF16, FP16])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("shape", [(16, 16), *FAST_TILES, "split", "last round 128", "last round 256"], ids=str)
def test_fast_sums(shape, glu, out_dtype):
    """Every shape by the 8-bit instruction: within its cut of the reference, and exact where no product is cut
    (whole numbers of at most 16 by 16: 2^8 by 1, nothing 2^-13 below)."""
    op = (M.MM_FP8_GLU if glu else M.MM_FP8) | M.FP8_FAST_SUMS
    if shape == "split":
        counts, N, K = [90, 0, 140], 72, 8192
    elif isinstance(shape, str):
        counts, N, K = split_sizes(glu, [1, 5, 9, 12, 24, 40], op, (128, 256) if shape.endswith("128") else (256, 128))
    else:
        counts, N, K = sizes_for(op, (shape[0], shape[1] // 2) if glu else shape, 1)
    x, xs, w, ws, first = _operands(counts, N, K, glu, seed=N)
    call = M.grouped_fp8_glu if glu else M.grouped_fp8_mm
    rows = torch.randperm(sum(counts), device="cuda", generator=_gen(4)).to(torch.int32)
    out = call(x, xs, w, ws, first, rows=rows, out_dtype=out_dtype, fast_sums=True)
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, rows, sum(counts))
    bound = fp8_bound(K, mag, top, True)
    if glu:
        (gate, up), (dg, du) = branches(ref, {}), branches(bound, {})
        assert_close(out, ref_act(gate, up, {}), act_bound(gate, up, dg, du, {}))
    else:
        assert_close(out, ref, bound)
        g = _gen(5)
        x = (torch.randint(-1, 2, x.shape, device="cuda", generator=g) * (torch.rand(x.shape, device="cuda", generator=g) < 200 / K)).float()
        w = torch.randint(-16, 17, w.shape, device="cuda", generator=g).float() * (torch.rand(w.shape, device="cuda", generator=g) < 0.1)
        x, w, xs, ws = x.to(E4M3), w.to(E4M3), torch.ones_like(xs), torch.ones_like(ws)
        ref = ref_fp8(x, xs, w, ws, first, rows, sum(counts))[0]
        assert 16 <= float(ref.abs().max()) <= 256
        assert torch.equal(call(x, xs, w, ws, first, rows=rows, out_dtype=out_dtype, fast_sums=True).double(), ref)


def test_fast_sums_of_random_products():
    """The cut's error where it is not the worst: each of an eight's products loses up to 2^-13 of the power of two
    of the largest, which is at most that product, either way: 2^-13 / sqrt(3) each, sqrt(8) of it an eight and
    sqrt(K / 8) of that a result, so 2^-13 / sqrt(3) sqrt(K) t with t the eights' rms largest product. Results and
    their rounding are as without the cut. (Three such errors are allowed.)"""
    counts, N, K = [1024], 1032, 4112
    x, xs, w, ws, first = _operands(counts, N, K, False, seed=1)
    xs, ws = torch.ones_like(xs), torch.ones_like(ws) * 2.0 ** -14
    out = M.fp8_mm(x, xs, w[0], ws[0], out_dtype=FP16, fast_sums=True).double()
    same = M.fp8_mm(x, xs, w[0], ws[0], out_dtype=FP16).double()
    ref, _, _, _ = ref_fp8(x, xs, w, ws, first, None, 1024)
    # the eights' largest products, of a sample of rows and columns
    px = (x.float()[:64, None] * w.float()[0, None, :64]).view(64, 64, K // 8, 8).abs().amax(-1) * 2.0 ** -14
    cut = 3 * 2.0 ** -13 / 3 ** 0.5 * K ** 0.5 * float(px.double().pow(2).mean()) ** 0.5
    rounding = float((ref.half().double() - ref).pow(2).mean()) ** 0.5
    assert float((same - ref).pow(2).mean()) ** 0.5 <= rounding * 1.001
    assert float((out - ref).pow(2).mean()) <= rounding ** 2 + cut ** 2
    assert abs(float((out - ref).mean())) <= cut / 50          # no lean to one side over a million results


def test_fast_sums_are_for_16_bit_results():
    x, xs, w, ws, first = _operands([40], 72, 272, False)
    for call in (lambda **k: M.fp8_mm(x, xs, w[0], ws[0], **k), lambda **k: M.grouped_fp8_mm(x, xs, w, ws, first, **k)):
        with pytest.raises(TypeError, match="fast_sums"):
            call(out_dtype=FP32, fast_sums=True)
        with pytest.raises(TypeError, match="fast_sums"):
            call(out=torch.empty(40, 72, device="cuda"), fast_sums=True)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = call(fast_sums=True)
        s.synchronize()
        assert torch.equal(call(fast_sums=True, stream=s), want)
        s.synchronize()


# ---- offsets that fall and overlap, where last rounds are in parts


@pytest.mark.parametrize("glu", [False, True])
def test_offsets_that_go_wrong_in_a_last_round(glu):
    """Three groups of rows 0 to 1200, to 2400 and, the offsets falling, 2000 to 4000, three groups of none: tiles
    enough for a last round in parts. Rows of one group are right, rows of none stay."""
    N, K, R = (2304 if glu else 4608), 4112, 4097
    op = M.MM_FP8_GLU if glu else M.MM_FP8
    rows, cols, parts = M.debug_mm_plan(op, 6, R, N, K)
    assert parts == 0 and last_round([1200, 1200, 0, 2000], N, rows, cols, -(-K // 128))[0] >= 2
    x, xs, w, ws, _ = _operands([R, 0, 0, 0, 0, 0], N, K, glu)
    first = torch.tensor([0, 1200, 2400, 2000, 4000, 1000, -7], dtype=torch.int32, device="cuda")
    out = torch.full((R, N), 7.5, dtype=BF16, device="cuda")
    (M.grouped_fp8_glu if glu else M.grouped_fp8_mm)(x, xs, w, ws, first, out=out)
    assert bool((out[4000:] == 7.5).all())
    for e, lo, hi in ((0, 0, 1200), (1, 1200, 2000), (3, 2400, 4000)):
        one = offsets([hi - lo])
        ref, mag, top, _ = ref_fp8(x[lo:hi], xs[lo:hi], w[e:e + 1], ws[e:e + 1], one, None, hi - lo)
        bound = fp8_bound(K, mag, top, False)
        if glu:
            (gate, up), (dg, du) = branches(ref, {}), branches(bound, {})
            assert_close(out[lo:hi], ref_act(gate, up, {}), act_bound(gate, up, dg, du, {}))
        else:
            assert_close(out[lo:hi], ref, bound)
