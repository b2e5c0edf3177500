"""lambda of differential attention and its gradient on a B200, against 64 bits."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import rf

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.mark.parametrize("heads,rows,dim,dtype", [(1, 1, 1, "fp32"), (7, 7, 33, "bf16"), (40, 40, 64, "fp32"), (6, 1, 64, "fp16"),
                                                  (33, 1, 7, "fp32"), (300, 300, 128, "fp16"), (2, 2, 1000, "bf16")])
def test_value_and_gradient(heads, rows, dim, dtype):
    gen = torch.Generator().manual_seed(heads + dim)
    vec = [(torch.randn(rows, dim, generator=gen) / dim ** 0.5).to(TYPES[dtype]).cuda() for _ in range(4)]
    dlam = torch.randn(heads, generator=gen).cuda()
    lam, grad = torch.empty(heads, device="cuda"), [torch.empty_like(v) for v in vec]
    rf.diff_lambda(*vec, 0.8, lam)
    rf.diff_lambda_backward(*vec, dlam, *grad)
    a, b, c, d = (v.double() for v in vec)
    e1, e2 = torch.exp((a * b).sum(1)), torch.exp((c * d).sum(1))
    # fp32: the dot products' chains of at most dim / 32 + 5 additions, expf (2 ulp) and the sums of at most heads terms
    step = 2.0 ** -24 * (dim / 32 + 16)
    e_dot = step * torch.stack([(a * b).abs().sum(1), (c * d).abs().sum(1)])
    r1, r2 = e_dot[0] + 2.0 ** -21, e_dot[1] + 2.0 ** -21
    want = (e1 - e2 + 0.8).expand(heads)
    tol = (e1 * r1 + e2 * r2 + 2.0 ** -23 * (e1 + e2 + 0.8)).expand(heads)
    assert ((lam.double() - want).abs() <= tol).all()
    g = dlam.double() if rows == heads else dlam.double().sum()[None]
    e_g = 0 * g if rows == heads else heads * 2.0 ** -24 * dlam.double().abs().sum()[None]
    u = torch.finfo(TYPES[dtype]).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    for got, e, r, other, sign in ((grad[0], e1, r1, b, 1), (grad[1], e1, r1, a, 1), (grad[2], e2, r2, d, -1), (grad[3], e2, r2, c, -1)):
        want = sign * (g * e)[:, None] * other
        err = ((g.abs() * r + e_g) * e)[:, None] * other.abs() + 2.0 ** -22 * want.abs()
        assert ((got.double() - want).abs() <= err + u * (want.abs() + err) + tiny).all()
