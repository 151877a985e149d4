"""8-bit floating-point products: that the tiles of a last round are split where the plan says so, for each type of
result, and sums that a cut or a lost term would change, on the GPU."""
import itertools

import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import act_bound, assert_close, branches, codes, fp8_bound, ref_act, ref_fp8
from products_util import BF16, FP16, FP32, offsets

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


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


def last_round(counts, N, K, rows, cols, glu):
    """(parts of each tile of the last round, sums that they leave in scratch) for tiles of rows x cols outputs at
    two blocks a CU: tiles in groups of eight row tiles over the columns, the last 512 or fewer of them in as many
    parts as fill 512 blocks, at most eight and of at least eight steps each; (1, 0) where they stay whole."""
    row_tiles = [min(rows, c - r) for c in counts for r in range(0, c, rows)]
    ptiles, steps = -(-N // cols), -(-K // 128)
    n = len(row_tiles) * ptiles
    rest = n % 512
    parts = min(512 // rest, 8, steps // 8) if rest else 1
    if parts < 2:
        return 1, 0
    words = 0
    for t in range(n - rest, n):
        grp, rem = divmod(t, 8 * ptiles)
        cur = min(8, len(row_tiles) - grp * 8)
        words += row_tiles[grp * 8 + rem % cur] * min(cols, N - rem // cur * cols)
    return parts, words * parts * (2 if glu else 1)


def split_sizes(glu, groups, op=None):
    """The least (counts, N, K) of a list that the plan takes in parts (0) and whose offsets make a last round that
    is split."""
    op = op or (M.MM_FP8_GLU if glu else M.MM_FP8)
    found = None
    for c, e, n, k in itertools.product([600, 1000, 1100, 2100, 4097], groups, [520, 1032, 2056, 2304, 4608], [2064, 4112, 7168]):
        counts = [c] if e == 1 else [c + 3, 0, c - 2] + [c] * (e - 3)
        if found is not None and sum(counts) * n * k >= found[0]:
            continue
        rows, cols, parts = M.debug_mm_plan(op, e, sum(counts), n, k)
        if parts == 0 and last_round(counts, n, k, rows, cols, glu)[0] >= 2:
            found = (sum(counts) * n * k, counts, n, k)
    assert found, "no such sizes"
    return found[1:]


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("groups", [[1], [5, 9, 12, 24, 40]])
@pytest.mark.parametrize("glu", [False, True])
def test_last_rounds_are_split_and_joined(glu, groups, out_dtype):
    """The plan's 0 parts, the tile count that the offsets make, and the sums that scratch (all ones before) holds
    afterwards agree, so the split and the join have run; and the results are right."""
    counts, N, K = split_sizes(glu, groups)
    op, R, E = M.MM_FP8_GLU if glu else M.MM_FP8, sum(counts), len(counts)
    rows, cols, parts = M.debug_mm_plan(op, E, R, N, K)
    assert parts == 0
    split, words = last_round(counts, N, K, rows, cols, glu)
    assert split >= 2
    x, xs, w, ws, first = _operands(counts, N, K, glu, seed=K)
    scratch = torch.full((M.mm_scratch_bytes(op, E, R, N, K),), 255, dtype=torch.uint8, device="cuda")
    call = M.grouped_fp8_glu if glu else M.grouped_fp8_mm
    out = call(x, xs, w, ws, first, out_dtype=out_dtype, scratch=scratch)
    assert int((scratch.view(torch.int32) != -1).sum()) == words
    ref, mag, top, _ = ref_fp8(x, xs, w, ws, first, None, R)
    bound = fp8_bound(K, mag, top, out_dtype != FP32)
    if glu:
        (gate, up), (dg, du) = branches(ref, {}), branches(bound, {})
        assert_close(out, ref_act(gate, up, {}), act_bound(gate, up, dg, du, {}))
    else:
        assert_close(out, ref, bound)
