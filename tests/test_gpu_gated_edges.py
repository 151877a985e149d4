"""The gated block where its activation's gradient saturates or its intermediate values leave their range, on the
GPU, elementwise against float64 with bounds derived here."""
import pytest
import torch

import block_scaled_fp4_histogram_amd as M
from gated_util import U, assert_close, joined
from products_util import BF16, FP16

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
