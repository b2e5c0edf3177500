"""SiLU of the group norm on fp32 tensors, on a B200: with gamma = 0 the activation's argument is beta itself."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import rf

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24                       # an fp32 operation
UNITS = 2.0 ** -22 + 2.0 ** -23         # ex2.approx and rcp.approx


@pytest.mark.parametrize("span", ["row", "sample"])
@pytest.mark.parametrize("width", [1024, 1023, 128, 33])
def test_silu_and_its_derivative_in_fp32(width, span):
    gen = torch.Generator().manual_seed(14)
    x = torch.randn(1, 1 if span == "row" else 2, 3, width, generator=gen).cuda()
    beta = torch.linspace(-80, 80, 3 * width).view(3, width).cuda()      # below -87 the result leaves fp32's normal range
    gamma = torch.zeros_like(beta)
    y, stats, ws = torch.empty_like(x), rf.group_norm_stats(x, span), rf.group_norm_workspace(x, span)
    rf.group_norm(x, gamma, beta, y, span=span, act="silu", stats=stats, ws=ws)
    dy = torch.zeros_like(x)
    dy[0, 0] = 1
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    rf.group_norm_backward(x, gamma, beta, dy, stats, dx, dgamma, dbeta, span=span, act="silu", ws=ws)
    z = beta.double()
    s = torch.sigmoid(z)
    # e^-z = 2^t, t = -z log2(e) as one product: its rounding (2^-24 |t|) and the constant's (2^-25.6) change 2^t by
    # |z| (2^-24 + 2^-26); then ex2, the sum with 1, the reciprocal
    e_s = z.abs() * (STEP + 2.0 ** -26) + UNITS + STEP
    want = z * s
    assert ((y.double() - want).abs() <= (e_s + STEP) * want.abs()).all()
    want = s * (1 + z * (1 - s))
    # 1 - s: s's error (an error e_s of e^-z changes s by e_s s (1 - s)) and its own rounding; then z, the sum, s
    tol = s * (z.abs() * (e_s * s * (1 - s) + (UNITS + 2 * STEP) * s + STEP) + STEP * (1 + z * (1 - s)).abs())
    tol = tol + (e_s + STEP) * want.abs()
    assert ((dbeta.double() - want).abs() <= tol).all(), float(((dbeta.double() - want).abs() / tol).max())
