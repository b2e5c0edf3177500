"""Short fp16 lists take P in two f16 parts: a tighter bound than one part can meet."""
import math

import pytest
import torch

from block_sparse_video_rearrange_b200 import rf
from tests import diff_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 160])
@pytest.mark.parametrize("rows", [16, 300, 1024])       # 1, 3 and 8 blocks
@pytest.mark.parametrize("d", [128, 64])
def test_maps_of_short_fp16_lists(d, rows, heads, monkeypatch):
    plan = rf.Plan([(rows, 0, 0, 0)], heads, heads, d, "BNSD", "fp16", 0.5)
    gen = torch.Generator().manual_seed(18)
    q, k, v = ((c * torch.randn(rows, d, generator=gen)).to(torch.float16).cuda() for c in (2, 2, 1))
    full = [x.expand(1, heads, rows, d).contiguous() for x in (q, k, v)]
    si, sn = plan.select_shapes()
    idx = torch.arange(si[2], dtype=torch.int32, device="cuda").expand(si).contiguous()
    num = torch.full(sn, si[2], dtype=torch.int32, device="cuda")
    lam = torch.full((heads,), 0.7, device="cuda")
    scale = 1 / math.sqrt(d // 2)
    b = rf.DiffBuffers(plan, train=True)
    rf.diff_attn(plan, *full, idx, num, lam, scale, b.o_r, b.ws, maps=b.maps, lse=b.lse)
    assert torch.equal(b.maps, b.maps[:, :, :1].expand_as(b.maps))
    # Two parts: what the second leaves of the first's rounding, 2^-11 of 2^-11 (and f16's smallest step, P_TINY).
    # fp32: scores of at most 64 in log2 units (checked), sums of |q k| alike, are off by 64 * 2^-22 = 2^-16; with ex2,
    # the sums of at most 1,024 terms (8 chains a block) and the products' accumulation by less than 2^-15.
    h = d // 2
    for w in (0, 1):
        size = scale * math.log2(math.e) * (q.double().abs()[:, w * h:w * h + h] @ k.double().abs()[:, w * h:w * h + h].T)
        assert size.max() <= 64
    monkeypatch.setattr(diff_ref, "P_STEP", 2.0 ** -22)
    monkeypatch.setattr(diff_ref, "FP32", 2.0 ** -15)
    one = rf.Plan([(rows, 0, 0, 0)], 1, 1, d, "BNSD", "fp16", 0.5)
    want = diff_ref.reference(one, *(x[:, :1] for x in full), idx[:, :1], num[:, :1], lam[:1], scale)
    for w in (0, 1):
        off = (b.maps[w, 0, 0].double() - want["maps"][w, 0]).abs()
        tol = want["maps_tol"][w, 0]
        assert (off <= tol).all(), float((off / tol).max())
