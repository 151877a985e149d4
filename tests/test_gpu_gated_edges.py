"""The gated block where its activation's gradient saturates or its intermediate values leave their range, on the
GPU, elementwise against float64 with bounds derived here."""
import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import U, assert_close, check_backward, check_forward, joined
from last_round_util import last_round
from products_util import BF16, FP16, offsets, ref_dx, ref_mm

pytestmark = pytest.mark.gpu


def _situ_grad(dh, gate, up):
    """(d gate, d up) of silu(4 tanh(gate / 4)) 25 tanh(up / 25) in float64, and the magnitudes of d gate's terms;
    1 - tanh^2 as 1 / cosh^2, which keeps its precision where the tanh is 1."""
    g, u = 4 * torch.tanh(gate / 4), 25 * torch.tanh(up / 25)
    s = torch.sigmoid(g)
    in_g, in_u = torch.cosh(gate / 4) ** -2, torch.cosh(up / 25) ** -2
    d = dh * u * s * in_g
    return d * (1 + g * (1 - s)), dh * g * s * in_u, (d * (1 + g.abs() * (1 - s))).abs()


@pytest.mark.parametrize("layout", [M.W13_UP_GATE, M.W13_GATE_UP])
@pytest.mark.parametrize("dtype,dh", [(BF16, 2.0 ** 30), (FP16, 2.0 ** 12)])
def test_situ_gradient_where_a_branch_saturates(dtype, dh, layout):
    """Gates to 60 and up branches to 500 either way: 1 - tanh^2 down to 4e-13 and 2e-17.

    1 - tanh^2(y) is 4 s (1 - s) of s = sigmoid(2 y): its two factors are good to 6 u each and to the rounding
    of 2 y (and of the constant in it), 2 |2 y| u more: |2 y| <= 40, 92 u at most. The rest of the product takes
    42 u more (tanh 8, the sigmoid 8 + 4 * 8, products): 2^-16 covers them."""
    v = torch.tensor([0.0, 0.5, 1.0, 3.0, 6.5, 12.0, 16.0, 18.0, 19.0, 20.5, 22.0, 24.0, 25.0, 27.0, 30.0, 34.0, 40.0, 60.0])
    v = torch.cat([v, -v])
    gate = v.repeat_interleave(40).view(len(v), 40)
    up = torch.tensor([0.0, 1.0, 10.0, 40.0, 80.0, 100.0, 110.0, 118.0, 122.0, 128.0, 135.0, 141.0, 150.0, 155.0, 170.0, 190.0,
                       230.0, 300.0, 400.0, 500.0])
    up = torch.cat([up, -up]).expand(len(v), 40)
    gate, up = gate.to(dtype).cuda(), up.to(dtype).cuda()
    form = dict(activation=M.ACT_SITU, layout=layout)
    d = torch.full_like(gate, dh)
    got = M.glu_grad(d, joined(gate, up, form), **form)
    rg, ru, mag = _situ_grad(d.double(), gate.double(), up.double())
    assert float(rg.abs().max()) > 0 and int((rg.abs() > 0).sum()) > 1000
    assert_close(got, joined(rg, ru, form), joined(mag, ru.abs(), form) * 2.0 ** -16 + 2.0 ** -100)


def test_situ_gradient_of_nan_and_infinite_projections():
    """NaN reaches both gradients from either branch; an infinite branch is a saturated one."""
    form = dict(activation=M.ACT_SITU)
    nan, inf = float("nan"), float("inf")
    gate = torch.tensor([nan, 1.0, inf, -inf, 1.0, 1.0, nan, 1.0], dtype=BF16, device="cuda")[None]
    up = torch.tensor([1.0, nan, 1.0, 1.0, inf, -inf, nan, 1.0], dtype=BF16, device="cuda")[None]
    got = M.glu_grad(torch.ones_like(gate), joined(gate, up, form), **form)
    dg, du = got[0, 8:], got[0, :8]
    assert dg.isnan().tolist() == du.isnan().tolist() == [True, True, False, False, False, False, True, False]
    assert dg[2:4].tolist() == [0.0, 0.0] and du[4:6].tolist() == [0.0, 0.0]
    rg, ru, _ = _situ_grad(1.0, torch.ones(1, dtype=torch.float64), torch.ones(1, dtype=torch.float64))
    at_cap = 1 / float(torch.tanh(torch.tensor(0.04, dtype=torch.float64)))     # 25 for up's 25 tanh(1 / 25)
    want = float(rg) * at_cap
    assert abs(float(dg[4]) - want) <= 2.0 ** -7 * want and abs(float(dg[5]) + want) <= 2.0 ** -7 * want


@pytest.mark.parametrize("alpha", [1.0, 1.702, -1.702, 1e30, -1e30, 1e-30, 0.0])
def test_gradient_where_alpha_gate_passes_the_range(alpha):
    """Gates to the ends of bf16 times alpha beyond fp32's range: the sigmoid is 0 or 1 there, and so is what the
    gradient has of it. dh and up + beta are 1, so d gate is sigmoid(z) (1 + z sigmoid(-z)), z = alpha gate, and
    d up the gated value; the sigmoid's error is within 16 u and 2 |z| u of it wherever it is not 0 (|z| < 90)."""
    v = torch.tensor([3.3e38, 2e38, 1e38, 1e30, 1e9, 60.0, 1.0, 0.0], dtype=torch.float64).to(BF16).double()
    gate = torch.cat([v, -v])[None].cuda()
    up = torch.zeros_like(gate)
    got = M.glu_grad(torch.ones_like(gate).to(BF16), joined(gate, up, {}).to(BF16), alpha=alpha, beta=1.0).double()
    z = float(torch.tensor(alpha, dtype=torch.float32)) * gate
    s, r = torch.sigmoid(z), torch.sigmoid(-z)
    rg, ru = s * (1 + z * r), gate * s
    units = (24 + 4 * z.abs().clamp(max=90)) * U
    assert_close(got[:, 16:].to(BF16), rg, units * s * (1 + (z * r).abs()) + 2.0 ** -120, "d gate")
    assert_close(got[:, :16].to(BF16), ru, units * ru.abs() + 2.0 ** -120 * (1 + gate.abs()), "d up")


# ---- last rounds in parts: offsets that go wrong, and two graphs at once

FALLING = [0, 1200, 2400, 2000, 4000, 1000, -7]      # rows 2000 to 2400 in two groups, from 4000 on in none
GLU, DX = (4097, 2304, 2056), (4097, 4360, 1032)     # rows, I, reduction


def _normal(seed, *shape, dtype=BF16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).mul_(scale).to(dtype)


def _splits(op, E, counts, I, reduction):
    """That a product of these sizes has a last round in parts."""
    R = GLU[0]
    rows, cols, parts = M.debug_mm_plan(op, E, R, *((reduction, I) if op == M.MM_GLU_DX else (I, reduction)))
    return parts == 0 and last_round(counts, I, rows, cols, -(-reduction // 64))[0] >= 2


def test_forward_with_offsets_that_go_wrong_in_a_last_round():
    """Rows of one group are right, rows of none stay, projections too."""
    R, I, K = GLU
    assert _splits(M.MM_GLU, 6, [1200, 1200, 0, 2000], I, K)
    x, w = _normal(1, R, K), _normal(2, 6, 2 * I, K, scale=K ** -0.5)
    h, pre = torch.full((R, I), 7.5, dtype=BF16, device="cuda"), torch.full((R, 2 * I), 7.5, dtype=BF16, device="cuda")
    M.grouped_glu(x, w, torch.tensor(FALLING, dtype=torch.int32, device="cuda"), out=h, pre=pre, limit=2.0)
    assert bool((h[4000:] == 7.5).all()) and bool((pre[4000:] == 7.5).all())
    for e, lo, hi in ((0, 0, 1200), (1, 1200, 2000), (3, 2400, 4000)):
        ref, mag, _ = ref_mm(x[lo:hi], w[e:e + 1], offsets([hi - lo]), None, hi - lo)
        check_forward(h[lo:hi], pre[lo:hi], ref, mag, K, dict(limit=2.0))


def test_backward_with_offsets_that_go_wrong_in_a_last_round():
    R, I, N = DX
    assert _splits(M.MM_GLU_DX, 6, [1200, 1200, 0, 2000], I, N)
    dy, w, pre = _normal(3, R, N), _normal(4, 6, N, I, scale=N ** -0.5), _normal(5, R, 2 * I, scale=2.0)
    d_pre, h = torch.full((R, 2 * I), 7.5, dtype=BF16, device="cuda"), torch.full((R, I), 7.5, dtype=BF16, device="cuda")
    M.grouped_glu_dx(dy, w, pre, torch.tensor(FALLING, dtype=torch.int32, device="cuda"), out=d_pre, h=h, limit=2.0)
    assert bool((d_pre[4000:] == 7.5).all()) and bool((h[4000:] == 7.5).all())
    for e, lo, hi in ((0, 0, 1200), (1, 1200, 2000), (3, 2400, 4000)):
        dh, mag, _ = ref_dx(dy[lo:hi].contiguous(), w[e:e + 1], offsets([hi - lo]))
        check_backward(d_pre[lo:hi], h[lo:hi], dh, (N + 1) * U * mag, pre[lo:hi], dict(limit=2.0))


def test_two_captured_last_rounds_replayed_at_once():
    """Two graphs on two streams, each with last rounds in parts forward and backward: their scratch is their own."""
    R, I, K = GLU
    _, I2, N = DX
    assert _splits(M.MM_GLU, 1, [R], I, K) and _splits(M.MM_GLU_DX, 1, [R], I2, N)
    first = offsets([R]).cuda()
    x, w = [_normal(s, R, K) for s in (1, 2)], [_normal(s, 1, 2 * I, K, scale=K ** -0.5) for s in (3, 4)]
    dy, wd = [_normal(s, R, N) for s in (5, 6)], [_normal(s, 1, N, I2, scale=N ** -0.5) for s in (7, 8)]
    pre = [_normal(s, R, 2 * I2, scale=2.0) for s in (9, 10)]

    def step(i):
        return M.grouped_glu(x[i], w[i], first), M.grouped_glu_dx(dy[i], wd[i], pre[i], first)

    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in (0, 1):
        step(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            outs.append(step(i))
    for turn in range(4):
        for i in (0, 1):                     # new inputs, and eager calls beside the replays
            x[i].copy_(_normal(20 + 2 * turn + i, R, K))
            dy[i].copy_(_normal(40 + 2 * turn + i, R, N))
        want = [[t.clone() for t in step(i)] for i in (0, 1)]
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
