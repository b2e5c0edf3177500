"""Differential attention on a B200 where parts of the tensors differ in size by many powers of two."""
import math

import pytest
import torch

from block_sparse_video_rearrange_b200 import rf
from tests import diff_ref

pytestmark = pytest.mark.gpu

GRADS = ("dq_r", "dk_r", "dv_r")


def grads(plan, q, k, v, do, idx, num, lam):
    b = rf.DiffBuffers(plan, train=True)
    b.lam.copy_(lam)
    scale = 1 / math.sqrt(plan.d // 2)
    rf.diff_attn(plan, q, k, v, idx, num, b.lam, scale, b.o_r, b.ws, maps=b.maps, lse=b.lse)
    rf.diff_attn_backward(plan, q, k, v, idx, num, b.lam, scale, b.maps, b.lse, do, b.dq_r, b.dk_r, b.dv_r, b.dlam, b.ws)
    rf.raise_on_device_fault(plan, b.ws, "test")
    return b


def fp16_layer(d, n1=4, n2=2, seqs=((70, 3, 16, 16), (300, 0, 0, 0)), keep=0.6):
    plan = rf.Plan(list(seqs), n1, n2, d, "TND", "fp16", 0.5)
    gen = torch.Generator().manual_seed(31)
    q, k, v = (torch.randn(plan.tensor_shape(h), generator=gen).to(torch.float16).cuda() for h in (n1, n2, n2))
    do = (2.0 ** -10 * torch.randn(plan.tensor_shape(n1), generator=gen)).to(torch.float16).cuda()   # a loss averaged over tokens
    idx, num = diff_ref.selection(plan, gen, keep)
    lam = 0.5 + 0.3 * torch.randn(n1, generator=gen)
    return plan, q, k, v, do, idx.cuda(), num.cuda(), lam.cuda()


# n1 = 4: each list over a cluster of CTAs; n1 = 96: one CTA a list
WIDTHS = [(128, 4, 2), (64, 4, 2), (128, 96, 24), (64, 96, 24)]


@pytest.mark.parametrize("d,n1,n2", WIDTHS)
def test_fp16_gradients_do_not_depend_on_v_that_nothing_lists(d, n1, n2):
    plan, q, k, v, do, idx, num, lam = fp16_layer(d, n1, n2)
    idx[idx == 1] = -1                                     # block 1 of each sequence: an unused slot in every list
    calm = grads(plan, q, k, v, do, idx, num, lam)
    for _, spans in diff_ref.block_rows(plan):
        r0, n = spans[1]
        v[r0:r0 + n] = 6e4
    loud = grads(plan, q, k, v, do, idx, num, lam)
    for nm in GRADS:
        assert torch.equal(getattr(calm, nm), getattr(loud, nm)), nm


@pytest.mark.parametrize("d,n1,n2", WIDTHS)
def test_fp16_gradients_of_a_sequence_do_not_depend_on_its_neighbour(d, n1, n2):
    plan, q, k, v, do, idx, num, lam = fp16_layer(d, n1, n2)
    first = int(plan.seq_info[0].length)
    calm = grads(plan, q, k, v, do, idx, num, lam)
    v[first:] *= 1000
    do[first:] *= 2.0 ** 10
    loud = grads(plan, q, k, v, do, idx, num, lam)
    for nm in GRADS:
        assert torch.equal(getattr(calm, nm)[:first], getattr(loud, nm)[:first]), nm


@pytest.mark.parametrize("d,n1,n2", WIDTHS)
def test_fp16_gradients_of_a_head_do_not_depend_on_other_groups(d, n1, n2):
    plan, q, k, v, do, idx, num, lam = fp16_layer(d, n1, n2)
    calm = grads(plan, q, k, v, do, idx, num, lam)
    rep = n1 // n2
    v[:, 0] *= 1000
    do[:, :rep] *= 2.0 ** 10
    lam[:rep] = 500.0
    loud = grads(plan, q, k, v, do, idx, num, lam)
    assert torch.equal(calm.dq_r[:, rep:], loud.dq_r[:, rep:])
    assert torch.equal(calm.dk_r[:, 1:], loud.dk_r[:, 1:]) and torch.equal(calm.dv_r[:, 1:], loud.dv_r[:, 1:])


@pytest.mark.parametrize("d,n1,n2", WIDTHS)
def test_fp16_gradients_of_a_row_do_not_depend_on_other_rows_of_do(d, n1, n2):
    """dQ: any other row's.  dK and dV: of query blocks that do not list the key block."""
    plan, q, k, v, do, idx, num, lam = fp16_layer(d, n1, n2)
    second, spans = diff_ref.block_rows(plan)[1]
    idx[second + 1][idx[second + 1] == 2] = -1             # the second sequence's block 1 does not list its block 2
    calm = grads(plan, q, k, v, do, idx, num, lam)
    row = spans[1][0] + 5
    do[row] *= 2.0 ** 14
    loud = grads(plan, q, k, v, do, idx, num, lam)
    rest = torch.arange(q.shape[0], device="cuda") != row
    assert torch.equal(calm.dq_r[rest], loud.dq_r[rest])
    r0, n = spans[2]
    for nm in ("dk_r", "dv_r"):
        assert torch.equal(getattr(calm, nm)[r0:r0 + n], getattr(loud, nm)[r0:r0 + n]), nm
        assert not torch.equal(getattr(calm, nm), getattr(loud, nm)), nm


@pytest.mark.parametrize("d", [128, 64])
def test_fp16_gradients_beside_a_large_value_elsewhere(d):
    """Against the formula, with bounds taken from each sequence on its own: the first one is small, the second large."""
    plan, q, k, v, do, idx, num, lam = fp16_layer(d)
    first = int(plan.seq_info[0].length)
    v[first:] *= 1000
    do[first:] *= 2.0 ** 10
    b = grads(plan, q, k, v, do, idx, num, lam)
    # the reference takes the power of two that dS carries from all that it is given: here from one sequence's rows
    alone_v, alone_do = v.clone(), do.clone()
    alone_v[first:], alone_do[first:] = 0, 0
    want = diff_ref.reference(plan, q, k, alone_v, idx, num, lam, 1 / math.sqrt(d // 2), alone_do)
    for nm in ("dq", "dk", "dv"):
        off = (getattr(b, nm + "_r")[:first].double() - want[nm][:first]).abs()
        tol = want[nm + "_tol"][:first]
        assert (off <= tol).all(), (nm, float((off / tol).max()))
