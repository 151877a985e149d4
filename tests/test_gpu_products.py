"""Ragged expert products, 8-bit integer products and route grouping on the GPU,
against float64 references elementwise (tests/products_util.py)."""
import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from products_util import (BF16, FP16, FP32, assert_int8, assert_product, gather, offsets, ref_dw, ref_dx, ref_group,
                           ref_int8, ref_mm, ref_quant)

pytestmark = pytest.mark.gpu

# group sizes around every tile height, empty groups in front, between and behind
COUNTS = {
    "one": [1],
    "few": [0, 1, 2, 0, 5, 1],
    "mixed": [0, 15, 16, 17, 0, 31, 33, 63, 64, 65, 1, 0],
    "large": [127, 0, 128, 129, 255, 256, 257, 3],
    "single": [300],
    "many": [(7 * i) % 5 for i in range(200)],
    "empty": [0, 0, 0],
}
SHAPES = [(8, 8), (72, 40), (136, 264), (256, 512), (1152, 320)]   # (N, K)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, dtype=BF16, scale=1.0):
    return torch.randn(*shape, device="cuda", generator=g).mul_(scale).to(dtype)


def _case(counts, N, K, dtype, gathered, seed=0):
    """x, w, dy, first, rows: rows repeat tokens, and some name none."""
    g = _gen(seed)
    R, E = sum(counts), len(counts)
    first = offsets(counts).cuda()
    T = max(1, R // 3) if gathered else R
    x, dy = _normal(g, T, K, dtype=dtype), _normal(g, R, N, dtype=dtype)
    w = _normal(g, E, N, K, dtype=dtype)
    rows = None
    if gathered:
        rows = torch.randint(0, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        if R > 3:
            rows[R // 2], rows[1], rows[-1] = -1, T, 2 ** 31 - 1
    return x, w, dy, first, rows


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out_dtype,gathered", [(BF16, BF16, False), (FP16, FP32, True)])
def test_forward_and_gradients(counts, N, K, dtype, out_dtype, gathered):
    x, w, dy, first, rows = _case(COUNTS[counts], N, K, dtype, gathered)
    R = dy.shape[0]
    out = M.grouped_mm(x, w, first, rows=rows, out_dtype=out_dtype)
    ref, mag, cov = ref_mm(x, w, first, rows, R)
    assert out.dtype == out_dtype and bool(cov.all())
    assert_product(out, ref, mag, K, "forward")
    dx = M.grouped_mm_dx(dy, w, first, out_dtype=out_dtype)
    ref, mag, _ = ref_dx(dy, w, first)
    assert_product(dx, ref, mag, N, "dx")
    dw = M.grouped_mm_dw(dy, x, first, rows=rows, out_dtype=out_dtype)
    ref, mag = ref_dw(dy, x, first, rows)
    assert_product(dw, ref, mag, max(COUNTS[counts]), "dw")


@pytest.mark.parametrize("T,k,E,N,K", [(8, 6, 384, 1152, 512), (2, 8, 256, 64, 2048), (1, 1, 1, 4608, 1024),
                                       (700, 2, 3, 520, 1040), (3000, 1, 2, 264, 136)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_routed_sizes(T, k, E, N, K, dtype):
    g = _gen(T)
    ids = torch.rand(T, max(E, k), device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    first, order, token, inverse = M.group_routes(ids, E)
    x, w = _normal(g, T, K, dtype=dtype), _normal(g, E, N, K, dtype=dtype)
    dy = _normal(g, T * k, N, dtype=dtype)
    out = M.grouped_mm(x, w, first, rows=token)
    ref, mag, cov = ref_mm(x, w, first, token, T * k)
    assert_product(out[cov], ref[cov], mag[cov], K, "forward")
    dx = M.grouped_mm_dx(dy, w, first)
    ref, mag, cov = ref_dx(dy, w, first)
    assert_product(dx[cov], ref[cov], mag[cov], N, "dx")
    dw = M.grouped_mm_dw(dy, x, first, rows=token, out_dtype=FP32)
    ref, mag = ref_dw(dy, x, first, token)
    assert_product(dw, ref, mag, T * k, "dw")


def test_gradients_match_differences():
    """dx and dw against central differences of sum(dy * forward): the product is linear in each
    operand, and with integers up to 4 every sum stays below 2^24, so all values are exact in fp32."""
    g = _gen(5)
    counts, N, K = [3, 0, 9, 20], 24, 40
    R, E = sum(counts), len(counts)
    first = offsets(counts).cuda()
    ints = lambda *s: torch.randint(-4, 5, s, device="cuda", generator=g).to(BF16)  # noqa: E731
    x, w, dy = ints(R, K), ints(E, N, K), ints(R, N)
    s = lambda xx, ww: (M.grouped_mm(xx, ww, first, out_dtype=FP32).double() * dy.double()).sum().item()  # noqa: E731
    dx = M.grouped_mm_dx(dy, w, first, out_dtype=FP32)
    dw = M.grouped_mm_dw(dy, x, first, out_dtype=FP32)
    for r, k in [(0, 0), (2, 39), (11, 17), (31, 8)]:
        up, down = x.clone(), x.clone()
        up[r, k] += 1
        down[r, k] -= 1
        assert (s(up, w) - s(down, w)) / 2 == dx[r, k].item()
    for e, n, k in [(0, 0, 0), (1, 3, 4), (2, 23, 39), (3, 12, 33)]:
        up, down = w.clone(), w.clone()
        up[e, n, k] += 1
        down[e, n, k] -= 1
        assert (s(x, up) - s(x, down)) / 2 == dw[e, n, k].item()


@pytest.mark.parametrize("N,K", [(72, 40), (264, 512)])
def test_rows_outside_the_groups_stay(N, K):
    counts, start, tail = [5, 0, 70, 140], 3, 9
    g = _gen(1)
    R = start + sum(counts) + tail
    first = offsets(counts, start).cuda()
    x, w, dy = _normal(g, R, K), _normal(g, 4, N, K), _normal(g, R, N)
    x[:start], x[-tail:], dy[:start], dy[-tail:] = float("nan"), float("inf"), float("inf"), float("nan")
    inside = slice(start, R - tail)
    for call, ref, width, terms in ((lambda o: M.grouped_mm(x, w, first, out=o), ref_mm(x, w, first, None, R), N, K),
                                    (lambda o: M.grouped_mm_dx(dy, w, first, out=o), ref_dx(dy, w, first), K, N)):
        out = torch.full((R, width), 7.5, dtype=BF16, device="cuda")
        call(out)
        assert_product(out[inside], ref[0][inside], ref[1][inside], terms)
        assert bool((out[:start] == 7.5).all()) and bool((out[-tail:] == 7.5).all())
    dw = M.grouped_mm_dw(dy, x, first)
    z = slice(start, R - tail)
    ref, mag = ref_dw(dy[z], x[z], first - start, None)
    assert_product(dw, ref, mag, R)


@pytest.mark.parametrize("N,K", [(72, 40), (264, 520), (40, 1032)])
def test_non_finite_values_stay_in_their_rows(N, K):
    """An infinity or NaN reaches the sums it is a term of and no other: not through a tile's padding
    rows, a partial last step of the reduction, nor another group's weights."""
    counts = [40, 0, 21, 3, 130]
    x, w, dy, first, _ = _case(counts, N, K, BF16, False, seed=3)
    R = dy.shape[0]
    x[7, K - 1], x[40, 0], w[1], dy[50, 3] = float("inf"), float("nan"), float("nan"), float("nan")
    ref, mag, _ = ref_mm(x, w, first, None, R)
    out = M.grouped_mm(x, w, first)
    ok = torch.ones(R, dtype=torch.bool, device="cuda")
    ok[7] = ok[40] = False
    assert_product(out[ok], ref[ok], mag[ok], K)
    assert bool(torch.isnan(out[40]).all()) and not bool(torch.isfinite(out[7]).any())
    ref, mag, _ = ref_dx(dy, w, first)
    out = M.grouped_mm_dx(dy, w, first)
    ok = torch.ones(R, dtype=torch.bool, device="cuda")
    ok[50] = False
    assert_product(out[ok], ref[ok], mag[ok], N)
    assert bool(torch.isnan(out[50]).all())
    ref, mag = ref_dw(dy, x, first, None)
    out = M.grouped_mm_dw(dy, x, first, out_dtype=FP32)
    fin = torch.isfinite(ref)
    assert bool((torch.isfinite(out) == fin).all())
    assert_product(out[fin], ref[fin], mag[fin], R)


def test_accumulated_weight_gradient():
    counts, N, K = [33, 0, 100], 136, 72
    x, w, dy, first, rows = _case(counts, N, K, BF16, True, seed=4)
    base = torch.randn(3, N, K, device="cuda", generator=_gen(9))
    out = base.clone()
    M.grouped_mm_dw(dy, x, first, rows=rows, out=out, accumulate=True)
    ref, mag = ref_dw(dy, x, first, rows)
    assert_product(out, ref + base.double(), mag + base.double().abs(), max(counts) + 1)
    assert torch.equal(out[1], base[1])


def test_offsets_that_go_wrong_stay_in_bounds():
    """Offsets outside [0, R] are clamped, groups that run backwards are empty."""
    g = _gen(2)
    R, N, K = 90, 72, 136
    x, w, dy = _normal(g, R, K), _normal(g, 3, N, K), _normal(g, R, N)
    first = torch.tensor([-5, 40, 30, 1000], dtype=torch.int32, device="cuda")
    fixed = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    got = M.grouped_mm(x, w, first)
    ref, mag, _ = ref_mm(x, w[[0, 2]], fixed, None, R)
    assert_product(got[:30], ref[:30], mag[:30], K)      # rows 30 .. 39 belong to groups 0 and 2
    assert_product(got[40:], ref[40:], mag[40:], K)
    dw = M.grouped_mm_dw(dy, x, first)
    assert bool((dw[1] == 0).all())


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 4112), (70, 256), (5, 7168), (300, 64)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantiser(rows, cols, dtype):
    g = _gen(rows)
    x = _normal(g, rows, cols, dtype=dtype)
    x *= torch.exp2(torch.randint(-10, 8, (rows, 1), device="cuda", generator=g)).to(dtype)
    x[:, 0] *= 50
    x[rows // 2] = 0
    q, s = M.quant_int8(x)
    rq, rs = ref_quant(x)
    assert torch.equal(s, rs) and torch.equal(q, rq)


def test_quantiser_on_ties_and_extreme_rows():
    cols = 256
    x = torch.zeros(8, cols, dtype=BF16)
    x[0, :255] = torch.arange(-127, 128) * 0.5      # amax 63.5: scale 0.5, every code exact
    x[1, 0], x[1, 1:64] = 127.0, torch.arange(63) + 0.5   # scale 1: ties go to even
    x[2, :3] = torch.tensor([2.0 ** -133, -(2.0 ** -132), 2.0 ** -127])  # subnormals
    x[3, :2] = torch.tensor([3.0e38, -1.0e38])
    x[4, 5], x[5, 6], x[6, 7] = float("inf"), float("nan"), float("-inf")
    x = x.cuda()
    q, s = M.quant_int8(x)
    rq, rs = ref_quant(x)
    assert torch.equal(torch.isnan(s), torch.isnan(rs)) and torch.equal(s.nan_to_num(), rs.nan_to_num())
    assert torch.equal(q, rq)
    assert q[1, 1:4].tolist() == [0, 2, 2]
    out = M.int8_mm(q, s, q, torch.ones(8, device="cuda"), out_dtype=FP32)
    assert bool(torch.isnan(out[4:7]).all()) and bool(torch.isfinite(out[:3]).all())   # row 3 overflows


@pytest.mark.parametrize("M_,N,K", [(1, 8, 16), (1, 4608, 7168), (5, 72, 48), (8, 4608, 1024), (16, 520, 272),
                                    (17, 264, 128), (33, 1032, 2064), (64, 256, 256), (129, 136, 400), (300, 640, 1024),
                                    (1025, 264, 144)])
@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32])
def test_int8_product(M_, N, K, out_dtype):
    g = _gen(M_)
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, w = i8(M_, K), i8(N, K)
    xs = torch.rand(M_, device="cuda", generator=g) + 0.1
    ws = (torch.rand(N, device="cuda", generator=g) + 0.1) / K / 100
    out = M.int8_mm(x, xs, w, ws, out_dtype=out_dtype)
    ref, _ = ref_int8(x, xs, w[None], ws[None], offsets([M_]).cuda(), None, M_)
    assert_int8(out, ref)


def test_int8_sums_are_exact_at_the_longest_reduction():
    K = 131056
    x = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    x[1] = 127
    w = torch.full((8, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(8, device="cuda")
    out = M.int8_mm(x, one[:2], w, one, out_dtype=FP32)
    assert out[0].tolist() == [float(16384 * K)] * 8
    want = torch.tensor(float(-16256 * K), dtype=torch.float64).float().item()
    assert out[1].tolist() == [want] * 8


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K,gathered", [(72, 48, True), (264, 528, False), (1152, 256, True)])
def test_grouped_int8_product(counts, N, K, gathered):
    c = COUNTS[counts]
    g = _gen(N)
    R, E = sum(c), len(c)
    T = max(1, R // 2) if gathered else R
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, w = i8(T, K), i8(E, N, K)
    xs, ws = torch.rand(T, device="cuda", generator=g) + 0.1, (torch.rand(E, N, device="cuda", generator=g) + 0.1) / K
    rows = None
    if gathered:
        rows = torch.randint(0, T, (R,), device="cuda", generator=g, dtype=torch.int32)
        if R > 2:
            rows[R // 2], rows[0] = -7, T
    first = offsets(c).cuda()
    out = M.grouped_int8_mm(x, xs, w, ws, first, rows=rows)
    ref, _ = ref_int8(x, xs, w, ws, first, rows, R)
    assert_int8(out, ref)


@pytest.mark.parametrize("T,k,E", [(0, 4, 8), (1, 1, 1), (8, 6, 384), (170, 6, 384), (171, 6, 384), (1024, 1, 3),
                                   (1025, 1, 1024), (4096, 8, 256), (333, 64, 17)])
def test_group_routes(T, k, E):
    g = _gen(T + k)
    ids = torch.randint(-2, E + 2, (T, k), device="cuda", generator=g, dtype=torch.int32)
    if T > 4:
        ids[T // 2:T // 2 + 2] = 2 ** 31 - 1
        ids[3] = -(2 ** 31)
    got = M.group_routes(ids, E)
    for a, b, name in zip(got, ref_group(ids.cpu(), E), ("first", "order", "token", "inverse")):
        assert torch.equal(a.cpu(), b), name


def test_group_routes_all_to_one_expert_and_none():
    for value in (2, -1):
        ids = torch.full((700, 3), value, dtype=torch.int32, device="cuda")
        for a, b in zip(M.group_routes(ids, 5), ref_group(ids.cpu(), 5)):
            assert torch.equal(a.cpu(), b)


def _train_step(x, ids, weights, w13, w2, dout):
    """A routed layer of 16-bit experts, forward and backward, from the entry points: the SwiGLU and
    the weighted sum over slots are torch's."""
    T, k = ids.shape
    E, N2, _ = w13.shape
    N = N2 // 2
    first, order, token, inverse = M.group_routes(ids, E)
    z = M.grouped_mm(x, w13, first, rows=token, out_dtype=FP32)
    up, gate = z[:, :N], z[:, N:]
    sg = torch.sigmoid(gate)
    h = (gate * sg * up).to(x.dtype)
    y = M.grouped_mm(h, w2, first, out_dtype=FP32)
    valid = inverse >= 0
    at = inverse.clamp(min=0).long()
    out = torch.where(valid[..., None], y[at] * weights[..., None], 0.0).sum(1)
    live = order >= 0
    wr = torch.where(live, weights.flatten()[order.clamp(min=0).long()], 0.0)
    dy = (dout[token.clamp(min=0).long()] * wr[:, None]).to(x.dtype)
    dw2 = M.grouped_mm_dw(dy, h, first, out_dtype=FP32)
    dh = M.grouped_mm_dx(dy, w2, first, out_dtype=FP32)
    dgate = dh * up * (sg + gate * sg * (1 - sg))
    dz = torch.cat([dh * gate * sg, dgate], 1).to(x.dtype)
    dw13 = M.grouped_mm_dw(dz, x, first, rows=token, out_dtype=FP32)
    dxr = M.grouped_mm_dx(dz, w13, first, out_dtype=FP32)
    dx = torch.where(valid[..., None], dxr[at], 0.0).sum(1)
    return out, dx, dw13, dw2


def _train_reference(x, ids, weights, w13, w2, dout):
    """The same layer in float64 by autograd, token by token's expert."""
    xd, a, b = (t.detach().double().cpu().requires_grad_() for t in (x, w13, w2))
    ids, wd = ids.cpu(), weights.double().cpu()
    E, N2, _ = a.shape
    out = torch.zeros(xd.shape[0], xd.shape[1], dtype=torch.float64)
    for e in range(E):
        t, j = ((ids == e).nonzero(as_tuple=True))
        z = xd[t] @ a[e].t()
        h = torch.nn.functional.silu(z[:, N2 // 2:]) * z[:, :N2 // 2]
        out = out.index_add(0, t, (h @ b[e].t()) * wd[t, j][:, None])
    out.backward(dout.double().cpu())
    return out.detach(), xd.grad, a.grad, b.grad


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_layer_of_16bit_experts_forward_and_backward(dtype):
    """The run of all products. Intermediates are rounded to 16 bits four times along the longest path
    (h, dy, dz and none on the fp32 outputs), each off by at most eps/2; the elementwise functions
    between them have slopes up to about 1.1 in both factors, so two products' worth of such errors
    stays within 8 half steps of each tensor's norm."""
    g = _gen(11)
    T, k, E, N, K = 150, 3, 7, 136, 264
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    ids[-4:] = -1
    ids[5, 1] = E + 3
    weights = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)
    x = _normal(g, T, K, dtype=dtype)
    w13, w2 = _normal(g, E, 2 * N, K, dtype=dtype, scale=K ** -0.5), _normal(g, E, K, N, dtype=dtype, scale=N ** -0.5)
    dout = torch.randn(T, K, device="cuda", generator=g)
    got = _train_step(x, ids, weights, w13, w2, dout)
    ref = _train_reference(x, ids, weights, w13, w2, dout)
    assert bool((got[0][-4:] == 0).all()) and bool((got[1][-4:] == 0).all())
    for name, a, b in zip(("out", "dx", "dw13", "dw2"), got, ref):
        rel = ((a.double().cpu() - b).norm() / b.norm()).item()
        assert rel <= 8 * torch.finfo(dtype).eps / 2, (name, rel)


def _int8_layer(x, ids, w13q, w13s, w2q, w2s):
    first, order, token, inverse = M.group_routes(ids, w13q.shape[0])
    xq, xs = M.quant_int8(x)
    z = M.grouped_int8_mm(xq, xs, w13q, w13s, first, rows=token, out_dtype=FP32)
    N = z.shape[1] // 2
    h = (torch.nn.functional.silu(z[:, N:]) * z[:, :N]).to(x.dtype)
    hq, hs = M.quant_int8(h)
    return M.grouped_int8_mm(hq, hs, w2q, w2s, first, out_dtype=FP32), first, token, hq, hs, z


def test_layer_of_int8_experts():
    """Each product of the run is held to its own definition on the inputs it got."""
    g = _gen(12)
    T, k, E, N, K = 90, 4, 6, 144, 272
    ids = torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32)
    x = _normal(g, T, K)
    w13q, w13s = M.quant_int8(_normal(g, E * 2 * N, K, scale=K ** -0.5))
    w2q, w2s = M.quant_int8(_normal(g, E * K, N, scale=N ** -0.5))
    w13q, w13s, w2q, w2s = w13q.view(E, 2 * N, K), w13s.view(E, 2 * N), w2q.view(E, K, N), w2s.view(E, K)
    y, first, token, hq, hs, z = _int8_layer(x, ids, w13q, w13s, w2q, w2s)
    xq, xs = ref_quant(x)
    assert_int8(z, ref_int8(xq, xs, w13q, w13s, first, token, T * k)[0])
    assert_int8(y, ref_int8(hq, hs, w2q, w2s, first, None, T * k)[0])


def test_captured_run_replays():
    """The whole run captured in one graph, two graphs sharing the caller's buffers, replayed with new
    inputs between eager calls: bit-identical to eager."""
    g = _gen(13)
    T, k, E, N, K = 64, 2, 5, 128, 256
    x, w13, w2 = _normal(g, T, K), _normal(g, E, 2 * N, K, scale=K ** -0.5), _normal(g, E, K, N, scale=N ** -0.5)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    weights, dout = torch.rand(T, k, device="cuda", generator=g), torch.randn(T, K, device="cuda", generator=g)
    args = (x, ids, weights, w13, w2, dout)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _train_step(*args)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = _train_step(*args)
        graphs.append((gr, outs))
    for rep in range(3):
        ids.copy_(torch.rand(T, E, device="cuda", generator=g).topk(k, dim=1).indices.to(torch.int32))
        x.copy_(_normal(g, T, K))
        if rep == 1:
            ids[10:] = -1
        want = [t.clone() for t in _train_step(*args)]
        torch.cuda.synchronize()
        for gr, outs in graphs:
            gr.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_results_repeat_and_other_streams():
    x, w, dy, first, rows = _case([0, 200, 3, 700], 264, 520, BF16, True, seed=6)
    ref = [M.grouped_mm(x, w, first, rows=rows), M.grouped_mm_dx(dy, w, first), M.grouped_mm_dw(dy, x, first, rows=rows)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = [M.grouped_mm(x, w, first, rows=rows, stream=side), M.grouped_mm_dx(dy, w, first, stream=side),
               M.grouped_mm_dw(dy, x, first, rows=rows, stream=side)]
        side.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_offsets_beyond_32_bits():
    """Weights, outputs and weight gradients past 2^31 elements: the last group's values are right."""
    E, N, K = 264, 1152, 7168
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda")
    g = _gen(8)
    w[-1] = _normal(g, N, K)
    counts = [0] * (E - 1) + [5]
    first = offsets(counts).cuda()
    x, dy = _normal(g, 5, K), _normal(g, 5, N)
    ref, mag, _ = ref_mm(x, w[-1:], offsets([5]).cuda(), None, 5)
    assert_product(M.grouped_mm(x, w, first), ref, mag, K)
    ref, mag, _ = ref_dx(dy, w[-1:], offsets([5]).cuda())
    assert_product(M.grouped_mm_dx(dy, w, first), ref, mag, N)
    M.grouped_mm_dw(dy, x, first, out=w)
    ref, mag = ref_dw(dy, x, offsets([5]).cuda(), None)
    assert_product(w[-1:], ref, mag, 5)
    assert not bool(w[:-1].any())
    del w
    R, N, K = 600000, 4096, 16
    x, w1 = _normal(g, R, K), _normal(g, 2, N, K)
    first = offsets([R - 7, 7]).cuda()
    out = M.grouped_mm(x, w1, first)
    ref, mag, _ = ref_mm(x[-100:], w1, offsets([93, 7]).cuda(), None, 100)
    assert_product(out[-100:], ref, mag, K)
    dx = M.grouped_mm_dx(out, w1, first)   # rows of out lie past 4 GiB
    ref, mag, _ = ref_dx(out[-100:], w1, offsets([93, 7]).cuda())
    assert_product(dx[-100:], ref, mag, N)
    rows = torch.arange(R - 1, -1, -1, device="cuda", dtype=torch.int32)
    dw = M.grouped_mm_dw(x, out, first, rows=rows, out_dtype=FP32)   # gathered rows past 4 GiB
    ref, mag = ref_dw(x, out, first, rows)
    assert_product(dw, ref, mag, R)


# sizes whose tiles would leave the chip idle: the reduction is split into parts joined by a second launch
SPLIT = [([70, 0, 200, 31], 264, 4104, 72), ([600], 136, 2600, 2608)]   # counts, N, K of forward, N of dx


@pytest.mark.parametrize("counts,N,K,Nx", SPLIT)
@pytest.mark.parametrize("dtype,out_dtype,gathered", [(BF16, BF16, True), (FP16, FP32, False)])
def test_split_reductions(counts, N, K, Nx, dtype, out_dtype, gathered):
    R, E = sum(counts), len(counts)
    assert M.mm_scratch_bytes(M.MM_FORWARD, E, R, N, K) > 0 and M.mm_scratch_bytes(M.MM_DX, E, R, 2608, N) > 0
    x, w, _, first, rows = _case(counts, N, K, dtype, gathered, seed=21)
    out = M.grouped_mm(x, w, first, rows=rows, out_dtype=out_dtype)
    ref, mag, _ = ref_mm(x, w, first, rows, R)
    assert_product(out, ref, mag, K, "forward")
    _, w, dy, first, _ = _case(counts, 2608, N, dtype, False, seed=22)
    dx = M.grouped_mm_dx(dy, w, first, out_dtype=out_dtype)
    ref, mag, _ = ref_dx(dy, w, first)
    assert_product(dx, ref, mag, 2608, "dx")


@pytest.mark.parametrize("gathered", [False, True])
def test_split_weight_gradient_accumulates(gathered):
    counts, N, K = [5000, 0, 3001], 72, 136
    R = sum(counts)
    assert M.mm_scratch_bytes(M.MM_DW, 3, R, N, K) > 0
    x, _, dy, first, rows = _case(counts, N, K, BF16, gathered, seed=23)
    ref, mag = ref_dw(dy, x, first, rows)
    assert_product(M.grouped_mm_dw(dy, x, first, rows=rows), ref, mag, max(counts))
    base = torch.randn(3, N, K, device="cuda", generator=_gen(24))
    out = base.clone()
    M.grouped_mm_dw(dy, x, first, rows=rows, out=out, accumulate=True)
    assert_product(out, ref + base.double(), mag + base.double().abs(), max(counts) + 1)
    assert torch.equal(out[1], base[1])


def test_split_products_leave_rows_outside_the_groups():
    counts, start, tail, N, K = [40, 200], 7, 11, 72, 4096
    R = start + sum(counts) + tail
    assert M.mm_scratch_bytes(M.MM_FORWARD, 2, R, N, K) > 0
    g = _gen(25)
    first = offsets(counts, start).cuda()
    x, w = _normal(g, R, K), _normal(g, 2, N, K)
    out = torch.full((R, N), -3.0, dtype=BF16, device="cuda")
    M.grouped_mm(x, w, first, out=out)
    ref, mag, cov = ref_mm(x, w, first, None, R)
    assert_product(out[cov], ref[cov], mag[cov], K)
    assert bool((out[~cov] == -3).all()) and int((~cov).sum()) == start + tail


@pytest.mark.parametrize("rows_given", [False, True])
def test_split_int8_product(rows_given):
    g = _gen(26)
    counts, N, K = [90, 0, 140], 136, 8192
    R = sum(counts)
    assert M.mm_scratch_bytes(M.MM_INT8, 3, R, N, K) > 0
    i8 = lambda *s: torch.randint(-128, 128, s, device="cuda", generator=g, dtype=torch.int8)  # noqa: E731
    x, w = i8(R, K), i8(3, N, K)
    xs, ws = torch.rand(R, device="cuda", generator=g), torch.rand(3, N, device="cuda", generator=g) / K
    rows = torch.randperm(R, device="cuda", generator=g).to(torch.int32) if rows_given else None
    first = offsets(counts).cuda()
    for dt in (BF16, FP32):
        out = M.grouped_int8_mm(x, xs, w, ws, first, rows=rows, out_dtype=dt)
        assert_int8(out, ref_int8(x, xs, w, ws, first, rows, R)[0])


def test_given_scratch_and_its_refusals():
    counts, N, K = [70, 200], 264, 4104
    x, w, _, first, _ = _case(counts, N, K, BF16, False, seed=27)
    need = M.mm_scratch_bytes(M.MM_FORWARD, 2, sum(counts), N, K)
    want = M.grouped_mm(x, w, first)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(M.grouped_mm(x, w, first, scratch=scratch), want)
    with pytest.raises(M.MoeError) as e:
        M.grouped_mm(x, w, first, scratch=scratch[:need - 16])
    assert e.value.code == M.MOE_ESCRATCH
    with pytest.raises(M.MoeError) as e:
        M.grouped_mm(x, w, first, scratch=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[4:])
    assert e.value.code == M.MOE_EINVAL
    with pytest.raises(M.MoeError) as e:                       # contiguous, but not 16-byte aligned
        M.grouped_mm(torch.empty(270 * K + 8, dtype=BF16, device="cuda")[1:270 * K + 1].view(270, K), w, first)
    assert e.value.code == M.MOE_EINVAL


def test_quantiser_on_more_rows_than_a_grid():
    """More rows than one grid of either kernel takes: every row of the ends and the turns between."""
    for rows, cols in ((1100000, 16), (300000, 8208)):
        x = torch.randn(rows, 16, device="cuda", generator=_gen(rows)).to(BF16).repeat(1, cols // 16)
        q, s = M.quant_int8(x)
        for at in (0, 262100, rows - 70):
            z = slice(at, at + 70)
            rq, rs = ref_quant(x[z])
            assert torch.equal(q[z], rq) and torch.equal(s[z], rs)
        assert torch.equal(s, (x[:, :16].float().abs().amax(1).double() / 127).float())


def test_two_products_at_once_on_two_streams():
    """Overlapping calls with scratch of their own."""
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    x, w, _, first, _ = _case([70, 0, 200], 264, 4104, BF16, False, seed=28)
    want = M.grouped_mm(x, w, first)
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs += [M.grouped_mm(x, w, first, stream=a), M.grouped_mm(x, w, first, stream=b)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("R,N,K", [(5, 72, 272), (200, 72, 272), (200, 136, 40)])
def test_x_without_rows(R, N, K):
    """Every product row then names no row: zeros, also where each kernel of the forward product runs."""
    first, rows = offsets([R // 2, R - R // 2]).cuda(), torch.full((R,), -1, dtype=torch.int32, device="cuda")
    x, w = torch.empty(0, K, dtype=BF16, device="cuda"), _normal(_gen(5), 2, N, K)
    out = M.grouped_mm(x, w, first, rows=rows, out=torch.full((R, N), 7.0, dtype=BF16, device="cuda"))
    assert not out.any()
    dw = M.grouped_mm_dw(_normal(_gen(6), R, N), x, first, rows=rows)
    assert not dw.any()
    if K % 16 == 0:
        wq, ws = M.quant_int8(w.view(2 * N, K))
        out = M.grouped_int8_mm(x.to(torch.int8), torch.empty(0, device="cuda"), wq.view(2, N, K), ws.view(2, N), first,
                                rows=rows, out=torch.full((R, N), 7.0, dtype=BF16, device="cuda"))
        assert not out.any()


def test_output_over_an_input_is_refused():
    x, w, first = _normal(_gen(7), 64, 64), _normal(_gen(8), 2, 64, 64), offsets([30, 34]).cuda()
    for call in (lambda: M.grouped_mm(x, w, first, out=x), lambda: M.grouped_mm_dx(x, w, first, out=x),
                 lambda: M.grouped_mm_dw(x, x, first, out=w[:, :, :], rows=w.view(-1).view(torch.int32)[:64])):
        with pytest.raises(M.MoeError, match="overlap"):
            call()


@pytest.mark.parametrize("cols", [16, 1024, 1040, 2064, 4096, 4112, 8208, 16384, 16400])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_quantiser_on_many_rows(cols, dtype):
    """Row counts past and no multiple of what a block takes, at each number of waves a row."""
    rows = 2051
    x = _normal(_gen(cols), rows, cols, dtype=dtype)
    x[1], x[700, cols - 1], x[rows - 1, 3] = 0, float("nan"), 300.0
    q, s = M.quant_int8(x)
    rq, rs = ref_quant(x)
    assert torch.equal(torch.isnan(s), torch.isnan(rs)) and torch.equal(s.nan_to_num(), rs.nan_to_num())
    assert torch.equal(q, rq)
