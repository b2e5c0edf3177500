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


# ---- V blocks of very different size ----------------------------------------------------------

def sized_layer(power, gap, heads, zero=False):
    """Text of five blocks; every row scores its target block 2^gap above the others, and the blocks' V are 1, 2^power,
    1, 2^-power and 1 (or 0) in size.  Rows of every block have every target."""
    d, blocks = 128, 5
    plan = rf.Plan([(128 * blocks, 0, 0, 0)], heads, heads, d, "BNSD", "bf16", 0.5)
    gen = torch.Generator().manual_seed(77)
    n = 128 * blocks
    q, k = (0.5 * torch.randn(n, d, generator=gen) for _ in range(2))
    code = math.sqrt(gap * 8 * math.log(2))                   # code^2 / 8 (the scale) is 2^gap in the exponential
    own = torch.arange(n) // 128
    target = torch.arange(n) % blocks
    for h in (0, 64):                                         # both maps
        q[torch.arange(n), h + target] += code
        k[torch.arange(n), h + own] += code
    v = torch.randn(n, d, generator=gen)
    v[128:256] *= 2.0 ** power
    v[384:512] *= 2.0 ** -power
    if zero:
        v[512:] = 0
    do = torch.randn(n, d, generator=gen)
    q, k, v, do = (x.to(torch.bfloat16).cuda().expand(1, heads, n, d).contiguous() for x in (q, k, v, do))
    si, sn = plan.select_shapes()
    idx = torch.arange(si[2], dtype=torch.int32, device="cuda").expand(si).contiguous()
    num = torch.full(sn, blocks, dtype=torch.int32, device="cuda")
    return plan, q, k, v, do, idx, num, torch.full((heads,), 0.7, device="cuda")


def sized_reference(q, k, v, do, lam, scale):
    """One dense head in 64 bits: {name: (value, bound)}.  As in diff_ref, but for P's smallest step in the forward product:
    f16's 2^-25, counted from the row's largest product of a probability and its block's largest |V|.  The backward pass
    makes P = 2^(s - lse) itself, in fp32, whose normal numbers end at 2^-126: a smaller P is 0 there, so P may be off by
    that much whatever its size (a score 130 below the row's largest, times a dA of 2^55, is a dS of 2^-75 that is lost
    beside the dS of 2^-55 of blocks as small as 2^-55)."""
    q, k, v, do = (x.double() for x in (q, k, v, do))
    u, step, fp32, least = 2.0 ** -8, diff_ref.P_STEP, diff_ref.FP32, 2.0 ** -126
    h = q.shape[1] // 2
    size = v.abs().view(-1, 128 * v.shape[1]).amax(1)
    size = torch.where(size > 0, 2.0 ** torch.ceil(torch.log2(size.clamp_min(1e-300))), 0.0)      # per block
    inv = torch.where(size > 0, 1 / size.clamp_min(1e-300), 0.0).repeat_interleave(128)
    p, o, e, lse = [], [], [], []
    for w in (0, 1):
        s = scale * (q[:, w * h:w * h + h] @ k[:, w * h:w * h + h].T)
        x = torch.softmax(s, 1)
        weight = (x * size.repeat_interleave(128)).amax(1, keepdim=True)
        p.append(x)
        o.append(x @ v)
        e.append((step + fp32) * (x @ v.abs()) + 2.0 ** -25 * weight * (v.abs() * inv[:, None]).sum(0))
        lse.append(torch.logsumexp(s, 1) / math.log(2.0))
    out, err = o[0] - lam * o[1], e[0] + abs(lam) * e[1]
    got = {"o": (out, u * (out.abs() + err) + err)}
    da, da_abs = do @ v.T, do.abs() @ v.abs().T
    a = p[0] - lam * p[1]
    a_err = u * a.abs() + (1 + u) * (fp32 * (p[0] + abs(lam) * p[1]) + least * (1 + abs(lam)))
    dv = a.T @ do
    got["dv"] = (dv, a_err.T @ do.abs())
    dq, dq_e, dk, dk_e = (torch.zeros_like(q) for _ in range(4))
    for w, c in ((0, 1.0), (1, -lam)):
        delta = (p[w] * da).sum(1, keepdim=True)
        ds = c * p[w] * (da - delta)
        d_err = (do.abs() * e[w]).sum(1, keepdim=True) + fp32 * (p[w] * da_abs).sum(1, keepdim=True)
        ds_e = u * ds.abs() + (1 + u) * abs(c) * (p[w] * (d_err + fp32 * (da_abs + delta.abs())) + least * (da_abs + delta.abs()))
        cols = slice(w * h, w * h + h)
        dq[:, cols], dq_e[:, cols] = scale * (ds @ k[:, cols]), scale * (ds_e @ k[:, cols].abs())
        dk[:, cols], dk_e[:, cols] = scale * (ds.T @ q[:, cols]), scale * (ds_e.T @ q[:, cols].abs())
    got["dq"], got["dk"] = (dq, dq_e), (dk, dk_e)
    for nm in ("dq", "dk", "dv"):
        x, t = got[nm]
        got[nm] = (x, t + u * (x.abs() + t))
    return got, lse


# heads = 1: the list over a cluster of CTAs; heads = 160: one CTA a list
@pytest.mark.parametrize("heads", [1, 160])
@pytest.mark.parametrize("power,gap,zero", [(18, 40, False), (24, 40, False), (30, 40, False), (30, 30, False), (30, 12, True),
                                            (40, 90, True), (55, 130, False), (20, 150, True)])
def test_rows_that_attend_to_small_v_beside_large(power, gap, zero, heads):
    plan, q, k, v, do, idx, num, lam = sized_layer(power, gap, heads, zero)
    b = grads(plan, q, k, v, do, idx, num, lam)
    want, lse = sized_reference(q[0, 0], k[0, 0], v[0, 0], do[0, 0], 0.7, 1 / 8)
    for nm, got in (("o", b.o_r), ("dv", b.dv_r), ("dk", b.dk_r), ("dq", b.dq_r)):
        assert torch.equal(got, got[:, :1].expand_as(got)), nm
        value, tol = want[nm]
        off = (got[0, 0].double() - value).abs()
        assert (off <= tol + 2.0 ** -120).all(), (nm, float((off / tol.clamp_min(1e-300)).max()))
    for w in (0, 1):
        assert ((b.lse[w, 0].double() - lse[w]).abs() <= 256 * 2.0 ** -22 + diff_ref.FP32).all()
    serve = rf.DiffBuffers(plan)
    serve.lam.copy_(lam)
    rf.diff_attn(plan, q, k, v, idx, num, serve.lam, 1 / 8, serve.o_r, serve.ws)
    assert torch.equal(serve.o_r, b.o_r)


# ---- scores of -infinity ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads,blocks", [(1, 5), (1, 12), (160, 5)])
def test_keys_whose_scores_are_minus_infinity_count_for_nothing(heads, blocks, dtype):
    """A block of such keys listed first, alone, or behind the others; a row without any other key is NaN, as softmax is."""
    d, n = 128, 128 * blocks
    plan = rf.Plan([(n, 0, 0, 0)], heads, heads, d, "BNSD", dtype, 0.5)
    gen = torch.Generator().manual_seed(8)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    q, k, v = (torch.randn(n, d, generator=gen) for _ in range(3))
    for c in (0, 64):                                          # both maps
        q[:, c] = q[:, c].abs() + 0.1
        k[:128, c] = k[-128:, c] = -float("inf")
    q, k, v = (x.to(dt).cuda().expand(1, heads, n, d).contiguous() for x in (q, k, v))
    lam = torch.full((heads,), 0.7, device="cuda")
    si, sn = plan.select_shapes()
    idx = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(si).contiguous()
    num = torch.full(sn, blocks, dtype=torch.int32, device="cuda")
    idx[1, :, 1:], num[1] = -1, 1                              # block 1 lists the first one alone
    idx[2, :, 0], idx[2, :, 1:], num[2] = blocks - 1, -1, 1    # block 2 the last one
    num[3] = 0                                                 # block 3 nothing
    b = rf.DiffBuffers(plan, train=True)
    rf.diff_attn(plan, q, k, v, idx, num, lam, 1 / 8, b.o_r, b.ws, maps=b.maps, lse=b.lse)
    rf.raise_on_device_fault(plan, b.ws, "test")
    assert torch.equal(b.o_r[:, :1].expand_as(b.o_r).isnan(), b.o_r.isnan())
    assert b.o_r[:, :, 128:384].isnan().all() and (b.o_r[:, :, 384:512] == 0).all()
    assert torch.isposinf(b.lse[:, :, 384:512]).all() and not torch.isposinf(b.lse[:, :, 128:384]).any()
    one = rf.Plan([(n, 0, 0, 0)], 1, 1, d, "BNSD", dtype, 0.5)
    keep = idx[:, :1].clone()
    keep[(keep == 0) | (keep == blocks - 1)] = -1              # the same without those keys
    keep[1:4] = -1
    want = diff_ref.reference(one, q[:, :1], k[:, :1].nan_to_num(neginf=0.0), v[:, :1], keep, num[:, :1], lam[:1], 1 / 8)
    rows = torch.ones(n, dtype=torch.bool, device="cuda")
    rows[128:512] = False
    off = (b.o_r[0].double() - want["o"][0]).abs()
    assert (off <= want["o_tol"][0])[:, rows].all(), float((off / want["o_tol"][0].clamp_min(1e-300))[:, rows].max())
