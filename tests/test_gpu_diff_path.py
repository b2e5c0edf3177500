"""Differential attention of whole layers through its user-level call, forward and backward, and with the group norm."""
import math

import pytest
import torch

from block_sparse_video_rearrange_b200 import diff, rf
from tests import diff_ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

LAYERS = {
    "bnsd": dict(seqs=[(100, 9, 17, 33)], layout="BNSD", dtype="bf16", batch=1, n1=3, n2=3, d=128, sparsity=0.6, order="tile"),
    "bnsd_gqa_pair": dict(seqs=[(20, 9, 16, 40)], layout="BNSD", dtype="fp16", batch=2, n1=4, n2=2, d=64, sparsity=0.7, order="frame_pair"),
    "tnd": dict(seqs=[(64, 9, 16, 32), (130, 3, 10, 19), (1, 0, 0, 0)], layout="TND", dtype="bf16", batch=1, n1=4, n2=2, d=128,
                sparsity=0.8, order="tile"),
}


def make(name, shared=False, vec_dtype=None):
    c = LAYERS[name]
    plan = rf.Plan(c["seqs"], c["n1"], c["n2"], c["d"], c["layout"], c["dtype"], c["sparsity"], batch=c["batch"], order=c["order"])
    gen = torch.Generator().manual_seed(11)
    dt = TYPES[c["dtype"]]
    q, k, v, w = (torch.randn(plan.tensor_shape(h), generator=gen).to(dt).cuda() for h in (c["n1"], c["n2"], c["n2"], c["n1"]))
    vec = [(0.2 * torch.randn(1 if shared else c["n1"], c["d"] // 2, generator=gen)).to(vec_dtype or torch.float32).cuda() for _ in range(4)]
    return c, plan, q, k, v, w, vec


def call(c, q, k, v, vec, **kw):
    return diff.rainfusion_diff_attention(q, k, v, c["seqs"], vec, 0.8, c["sparsity"], c["layout"], order=c["order"], **kw)


def selection(c, plan, q, k, v):
    """The selection that the call makes: the plan's ranking is deterministic."""
    b = rf.Buffers(plan)
    rf.rearrange(plan, q, k, v, b.q_r, b.k_r, b.v_r, b.ws)
    rf.pool_select(plan, None, None, b.select_idx, b.select_num, b.ws)
    return b


def to_original(plan, x, heads):
    """A rearranged 64-bit tensor back in original token order, by the plan's host-side permutation."""
    out = torch.empty_like(x)
    if plan.layout == "BNSD":
        out[:, :, torch.from_numpy(plan.permutation()).to(x.device)] = x
        return out
    for i, s in enumerate(plan.seq_info):
        r0 = int(s.row_offset)
        out[r0 + torch.from_numpy(plan.permutation(i)).to(x.device)] = x[r0:r0 + int(s.length)]
    return out


def within(got, want, tol, what):
    off = (got.double() - want).abs()
    assert (off <= tol).all(), (what, float((off / tol.clamp_min(1e-300)).max()))


@pytest.mark.parametrize("shared,vec_dtype", [(False, torch.float32), (True, torch.bfloat16)])
@pytest.mark.parametrize("name", list(LAYERS))
def test_layer_and_its_gradients(name, shared, vec_dtype):
    c, plan, q, k, v, w, vec = make(name, shared, vec_dtype)
    for t in (q, k, v, *vec):
        t.requires_grad_()
    o = call(c, q, k, v, vec)
    o.backward(w)
    with torch.no_grad():
        assert torch.equal(call(c, q, k, v, vec), o)
        b = selection(c, plan, q, k, v)
        do_r = torch.empty_like(q)
        rf.rearrange_rows(plan, w, do_r)
        a, bb, cc, dd = (t.double() for t in vec)
        e1, e2 = torch.exp((a * bb).sum(1)), torch.exp((cc * dd).sum(1))
        lam = (e1 - e2 + 0.8).expand(plan.n1)
        want = diff_ref.reference(plan, b.q_r, b.k_r, b.v_r, b.select_idx, b.select_num, lam, 1 / math.sqrt(plan.d // 2), do_r)
        # lambda itself is an fp32 number: its rounding and that of its exponentials, at most 2^-19 here
        dlam_err = 2.0 ** -19
        for nm, got in (("o", o), ("dq", q.grad), ("dk", k.grad), ("dv", v.grad)):
            val, tol = (to_original(plan, want[x], 0) for x in (nm, nm + "_tol"))
            within(got, val, tol + dlam_err * val.abs().max(), nm)
        g = want["dlam"].sum()[None] if shared else want["dlam"]
        ge = want["dlam_tol"].sum()[None] if shared else want["dlam_tol"]
        u = torch.finfo(vec_dtype).eps / 2
        for t, e, other, sign in ((vec[0], e1, bb, 1), (vec[1], e1, a, 1), (vec[2], e2, dd, -1), (vec[3], e2, cc, -1)):
            val = sign * (g * e)[:, None] * other
            err = (ge * e)[:, None] * other.abs() + 2.0 ** -18 * (val.abs() + (g.abs() * e)[:, None] * other.abs())
            within(t.grad, val, err + u * (val.abs() + err), "vectors")


@pytest.mark.parametrize("name,span,act", [("bnsd", "row", "none"), ("bnsd_gqa_pair", "sample", "silu"), ("tnd", "row", "silu"),
                                           ("tnd", "sample", "none")])
def test_layer_with_group_norm_equals_its_parts(name, span, act):
    """The norm of the layer's own output, on its own view of each layout; gradients through both."""
    c, plan, q, k, v, w, vec = make(name)
    gen = torch.Generator().manual_seed(2)
    gamma, beta = (1 + 0.1 * torch.randn(plan.n1, plan.d, generator=gen)).cuda(), (0.1 * torch.randn(plan.n1, plan.d, generator=gen)).cuda()
    leaves = [q, k, v, *vec, gamma, beta]
    for t in leaves:
        t.requires_grad_()
    y = call(c, q, k, v, vec, norm=(gamma, beta), norm_span=span, norm_act=act)
    assert y.shape == q.shape
    got = torch.autograd.grad(y, leaves, w)
    o = call(c, q, k, v, vec).detach().requires_grad_()
    x = o.transpose(1, 2) if plan.layout == "BNSD" else o[None]
    rows = [int(s.length) for s in plan.seq_info] if plan.layout == "TND" and span == "sample" else [x.shape[1]]
    outs = []
    for part in x.double().split(rows, dim=1):         # the formula in 64 bits
        dims = (3,) if span == "row" else (1, 3)
        mu = part.mean(dims, keepdim=True)
        z = gamma.double() * (part - mu) / ((part - mu).pow(2).mean(dims, keepdim=True) + 1e-5).sqrt() + beta.double()
        outs.append(z * torch.sigmoid(z) if act == "silu" else z)
    want = torch.cat(outs, 1)
    want = want.transpose(1, 2) if plan.layout == "BNSD" else want[0]
    u = torch.finfo(q.dtype).eps / 2
    # one rounding of y; fp32 in between (rows of O can be small beside the group's mean: 2^-12 of the largest |y|)
    assert ((y.double() - want).abs() <= u * want.abs() + 2.0 ** -12 * want.abs().amax()).all()
    do, dg, db = torch.autograd.grad(want, [o, gamma, beta], w.double())
    # gradients of gamma and beta: fp32 sums over all rows of terms that carry y's fp32 error
    for a, b in ((got[-2], dg), (got[-1], db)):
        assert (a - b).abs().max() <= 2.0 ** -10 * b.abs().max()
    # the layer's gradients: exactly those of the layer called with the norm's dx
    o2 = call(c, q, k, v, vec)
    x2 = o2.transpose(1, 2) if plan.layout == "BNSD" else o2[None]
    dx = []
    for xp, wp in zip(x2.detach().split(rows, 1), (w.transpose(1, 2) if plan.layout == "BNSD" else w[None]).split(rows, 1)):
        xp = xp.requires_grad_()
        dx.append(torch.autograd.grad(diff.group_norm(xp, gamma, beta, span=span, act=act), xp, wp)[0])
    dx = torch.cat(dx, 1)
    assert ((dx.double() - (do.transpose(1, 2) if plan.layout == "BNSD" else do[None]).double()).abs()
            <= u * dx.double().abs() + 2.0 ** -8 * dx.double().abs().max()).all()
    parts = torch.autograd.grad(x2, [q, k, v, *vec], dx)
    for a, b in zip(got, parts):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """The kernels' gradients against central differences of the 64-bit layer with the same selection."""
    c, plan, q, k, v, w, vec = make("bnsd")
    for t in (q, k, v):
        t.requires_grad_()
    call(c, q, k, v, vec).backward(w)
    b = selection(c, plan, q, k, v)
    lam = torch.exp((vec[0] * vec[1]).sum(1)) - torch.exp((vec[2] * vec[3]).sum(1)) + 0.8
    w_r = torch.empty_like(w)
    rf.rearrange_rows(plan, w, w_r)
    base = [x.double() for x in (b.q_r, b.k_r, b.v_r)]


    def loss(xs):
        # reference() reads the type of q for its bounds only
        out = diff_ref.reference(plan, *(x for x in xs), b.select_idx, b.select_num, lam, 1 / math.sqrt(plan.d // 2))
        return float((out["o"] * w_r.double()).sum())
    gen = torch.Generator("cuda").manual_seed(9)
    for i, t in enumerate((q, k, v)):
        g_r = torch.empty_like(t)
        rf.rearrange_rows(plan, t.grad, g_r)
        way = torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * way, base[i] - h * way
        slope = (loss(up) - loss(down)) / (2 * h)
        mine = float((g_r.double() * way).sum())
        # bf16 gradients: each of N elements off by about 2^-8 of itself at random signs, 6 standard deviations
        spread = 2.0 ** -8 * float((g_r.double() * way).pow(2).sum().sqrt()) * 6
        assert abs(slope - mine) <= spread + 1e-4 * abs(slope), (i, slope, mine)


def test_group_norm_of_a_feature_map():
    """[batch, rows, channels] with num_groups, broadcast and non-contiguous inputs, and an expanded gradient."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(3, 50, 24, generator=gen).cuda().requires_grad_()
    gamma, beta = torch.rand(24, generator=gen).cuda().requires_grad_(), torch.randn(24, generator=gen).cuda().requires_grad_()
    y = diff.group_norm(x, gamma, beta, num_groups=6, act="silu")
    want = torch.nn.functional.silu(torch.nn.functional.group_norm(x.double().transpose(1, 2), 6, gamma.double(), beta.double(), 1e-5)).transpose(1, 2)
    assert y.shape == x.shape and (y - want).abs().max() <= 2e-6 * want.abs().max() + 2e-6
    got, ref = torch.autograd.grad(y.sum(), [x, gamma, beta]), torch.autograd.grad(want.sum(), [x, gamma, beta])
    for a, b in zip(got, ref):
        assert (a - b).abs().max() <= 2.0 ** -15 * max(1.0, float(b.abs().max())) * 4
    one = torch.randn(1, 50, 24, generator=gen).cuda().requires_grad_()
    y = diff.group_norm(one.expand(3, 50, 24), gamma, beta, num_groups=6)
    g = torch.autograd.grad(y.square().sum(), one)[0]
    y1 = diff.group_norm(one, gamma, beta, num_groups=6)
    g1 = torch.autograd.grad(y1.square().sum(), one)[0]
    assert torch.equal(y[1], y1[0]) and (g - 3 * g1).abs().max() <= 2.0 ** -20 * max(1.0, float(g1.abs().max())) * 8
    t = torch.randn(3, 24, 50, generator=gen).cuda().transpose(1, 2)        # channels first in memory
    assert torch.equal(diff.group_norm(t, gamma, beta, num_groups=6), diff.group_norm(t.contiguous(), gamma, beta, num_groups=6))


def test_a_layer_in_a_graph_without_gradients_and_refusals():
    c, plan, q, k, v, w, vec = make("bnsd")
    want = call(c, q, k, v, vec)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(RuntimeError):
            call(c, q, k, v, vec)                      # check=True would synchronise
        with pytest.raises(RuntimeError):
            call(c, q.detach().requires_grad_(), k, v, vec, check=False)
        o = call(c, q, k, v, vec, check=False, plan=plan)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want)


def test_tensors_made_on_another_stream():
    c, plan, q, k, v, w, vec = make("tnd")
    want = call(c, q, k, v, vec)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q2 = q + 0
        q2.requires_grad_()
        o = call(c, q2, k, v, vec)
        o.backward(w)
    torch.cuda.current_stream().wait_stream(side)
    q.requires_grad_()
    call(c, q, k, v, vec).backward(w)
    assert torch.equal(o, want) and torch.equal(q.grad, q2.grad)
