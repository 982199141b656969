"""SiLU*mul and its gradient over the whole range of finite operands, and over sizes of every way of storing."""
import itertools

import pytest
import torch

import moe_w4a16_grouped_amd as moe
from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def _references(g, u, d):
    """(h, dg, du) and the errors of the first two factors' arithmetic, in 64 bits; s below 2^-126 counts as 0."""
    s = torch.sigmoid(g)
    s = torch.where(s < 2.0 ** -126, 0, s)
    exp_err = 2.0 ** -18 + g.abs().clamp(max=88) * 2.0 ** -23  # fast exponential and quotient, argument rounding
    es = exp_err * s + 2.0 ** -24
    h, dg, du = g * s * u, d * u * s * (1 + g * (1 - s)), d * g * s
    # as for moderate operands; where s is 0 the result is an exact 0, and beyond |g| = 88 so is s or 1 - s
    slope = s * (g.abs().clamp(max=88) * es + 2.0 ** -22 * (1 + g.abs().clamp(max=88)))
    return h, dg, du, exp_err * h.abs(), exp_err * dg.abs() + (d * u).abs() * slope, exp_err * du.abs()


def _check(got, ref, err, label):
    top = torch.finfo(got.dtype).max
    over = ref.abs() > top * (1 + ru.HALF_STEP[got.dtype])
    assert not torch.isnan(got).any(), label
    assert bool((got[over].double() == torch.sign(ref[over]) * float("inf")).all()), label
    ru.assert_close(got[~over], ref[~over], err[~over], label)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_large_and_small_finite_operands(dtype):
    """Products of two operands may pass fp32 where the result does not: no NaN, no infinity, no lost small factor."""
    wide = dtype == BF16
    gs = [0.0, 1.0, -1.0, -1.28125, 20.0, -20.0, 80.0, -80.0, 90.0, -90.0, -110.0] + ([1e20, -1e20, 3.3e38, -3.3e38] if wide else [6e4, -6e4])
    vs = [1.0, -3.0, 0.0] + ([1e-30, 1e-20, -1e10, 1e20, -1e20, 3.3e38] if wide else [1e-6, 6e4, -6e4])
    grid = list(itertools.product(gs, vs, vs))
    grid += [grid[-1]] * (-len(grid) % 8)
    g, u, d = (torch.tensor(c, dtype=torch.float64).to(dtype).cuda()[None] for c in zip(*grid))
    G = torch.cat([g, u], dim=1)
    h, dg, du, eh, eg, eu = _references(g.double(), u.double(), d.double())
    _check(moe.moe_silu_mul(G), h, eh, "h")
    dG = moe.moe_silu_mul_grad(G, d)
    _check(dG[:, :g.shape[1]], dg, eg, "dg")
    _check(dG[:, g.shape[1]:], du, eu, "du")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R,I", [(700, 6152), (2731, 2056)])
def test_results_of_some_megabytes(R, I, dtype):
    """Results too large for the L2s whose operands still lie in the memory-side cache."""
    gen = torch.Generator(device="cuda").manual_seed(R)
    G = (torch.randn((R, 2 * I), generator=gen, device="cuda") * 3).to(dtype)
    d = torch.randn((R, I), generator=gen, device="cuda").to(dtype)
    assert 8 << 20 < R * I * 2 and R * I * 6 < 256 << 20
    g, u = G.double().chunk(2, dim=1)
    h, dg, du, eh, eg, eu = _references(g, u, d.double())
    ru.assert_close(moe.moe_silu_mul(G), h, eh, "h")
    ru.assert_close(moe.moe_silu_mul_grad(G, d), torch.cat([dg, du], dim=1), torch.cat([eg, eu], dim=1), "dG")
