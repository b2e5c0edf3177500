"""Group norm on a B200 with infinities in its input."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import rf

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("span", ["row", "sample"])
@pytest.mark.parametrize("rows,width", [(1, 16), (700, 16), (700, 10), (61, 1000)])
def test_an_infinity_makes_its_group_nan_and_no_other(rows, width, span, dtype, value):
    """Mean and variance of a group with an infinity do not exist, wherever it lies (the first row, a lane's first row,
    the last, any slice)."""
    gen = torch.Generator().manual_seed(12)
    clean = torch.randn(2, rows, 3, width, generator=gen).to(dtype).cuda()
    gamma, beta = (torch.randn(3, width, generator=gen).cuda() for _ in range(2))
    want = torch.empty_like(clean)
    rf.group_norm(clean, gamma, beta, want, span=span)
    for r in sorted({0, 1, 7, 33, rows // 2, rows - 2, rows - 1}):
        if not 0 <= r < rows:
            continue
        for c in (0, width - 1):
            x, y = clean.clone(), torch.empty_like(clean)
            x[1, r, 1, c] = value
            rf.group_norm(x, gamma, beta, y, span=span)
            hit = torch.zeros_like(x, dtype=torch.bool)
            if span == "row":
                hit[1, r, 1] = True
            else:
                hit[1, :, 1] = True
            assert torch.equal(torch.isnan(y), hit), (r, c)
            assert torch.equal(y[~hit], want[~hit]), (r, c)
