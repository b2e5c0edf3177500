"""Group norm with an activation on a B200 against its formula in 64 bits, with bounds from the fp32 steps in between."""
import pytest
import torch

from block_sparse_video_rearrange_b200 import diff, rf

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# batch, rows, groups, width, dtype, params, span, act, how the rows lie, offset of the values
CASES = {
    "one_value": (1, 1, 1, 1, "fp32", "fp32", "row", "none", "last", 0.0),
    "one_row": (1, 1, 3, 128, "bf16", "fp32", "row", "silu", "last", 0.5),
    "heads_tnd": (1, 1000, 5, 128, "bf16", "fp32", "row", "none", "last", 1.0),
    "heads_bnsd": (2, 333, 4, 64, "fp16", "fp16", "row", "silu", "headmajor", 1.0),
    "odd_width": (2, 50, 3, 33, "bf16", "bf16", "row", "silu", "last", -2.0),
    "wide_row": (1, 37, 2, 1000, "bf16", "fp32", "row", "none", "last", 0.0),
    "wide_odd_row": (1, 9, 2, 1023, "fp32", "fp32", "row", "silu", "last", 3.0),
    "full_width": (1, 9, 1, 1024, "fp16", "fp32", "row", "none", "last", 0.0),
    "narrow": (3, 40, 7, 4, "fp32", "fp32", "row", "none", "last", 0.0),
    "two_wide": (1, 11, 2, 2, "fp16", "fp32", "row", "silu", "last", 0.0),
    "padded_rows": (2, 129, 3, 64, "bf16", "fp32", "row", "none", "padded", 0.0),
    "s_one_row": (2, 1, 2, 16, "bf16", "fp32", "sample", "silu", "last", 0.0),
    "s_odd_width": (2, 700, 32, 10, "bf16", "bf16", "sample", "silu", "last", 1.0),
    "s_scalar": (1, 97, 3, 33, "fp16", "fp32", "sample", "none", "last", 0.0),
    "s_headmajor": (2, 1500, 3, 64, "fp16", "fp32", "sample", "silu", "headmajor", 1.0),
    "s_far_mean": (1, 2000, 2, 8, "fp32", "fp32", "sample", "none", "last", 300.0),
    "s_wide": (1, 61, 2, 1500, "fp32", "fp32", "sample", "none", "last", 0.0),
    "s_wide_bf16": (1, 33, 1, 5000, "bf16", "fp32", "sample", "silu", "last", 0.0),
    "s_padded": (3, 257, 4, 24, "bf16", "bf16", "sample", "silu", "padded", 0.0),
}


def make(name, seed=0):
    batch, rows, groups, width, dt, pt, span, act, lie, offset = CASES[name]
    gen = torch.Generator().manual_seed(seed + 7)
    shape = (batch, rows, groups, width)

    def lay(x):
        x = x.to(TYPES[dt]).cuda()
        if lie == "headmajor":
            return x.transpose(1, 2).contiguous().transpose(1, 2)
        if lie == "padded":     # rows further apart than they are long
            pad = torch.full((batch, rows, groups + 1, width), float("nan"), dtype=x.dtype, device="cuda")
            pad[:, :, :groups] = x
            return pad[:, :, :groups]
        return x
    x = lay(torch.randn(shape, generator=gen) + offset)
    dy = lay(torch.randn(shape, generator=gen))
    gamma = (1 + 0.2 * torch.randn(groups, width, generator=gen)).to(TYPES[pt]).cuda()
    beta = (0.3 * torch.randn(groups, width, generator=gen)).to(TYPES[pt]).cuda()
    return x, dy, gamma, beta, span, act


def reference(x, dy, gamma, beta, span, act, eps):
    """Values and bounds.  fp32 sums: at most 2^9 additions in a row on any path (2^-15 of the summed magnitudes);
    sigmoid from the fast exponential and one division: 2^-19 relative."""
    chain, sig = 2.0 ** -15, 2.0 ** -19
    u, pu = torch.finfo(x.dtype).eps / 2, torch.finfo(gamma.dtype).eps / 2
    dims = (3,) if span == "row" else (1, 3)
    xd, gm, bt, up = x.double(), gamma.double(), beta.double(), dy.double()

    def mean(t):
        return t.mean(dims, keepdim=True)
    mu = mean(xd)
    sd = (mean((xd - mu) ** 2) + eps).sqrt()
    xh = (xd - mu) / sd
    # the mean is summed about 0 (rows) or a value of the data (samples); either way at most about max |x|
    e_xh = (chain * xd.abs().amax(dims, keepdim=True) + 2.0 ** -23 * xd.abs()) / sd + 2 * chain * xh.abs()
    z = gm * xh + bt
    e_z = gm.abs() * e_xh + 2.0 ** -22 * ((gm * xh).abs() + bt.abs())
    if act == "silu":
        s = torch.sigmoid(z)
        y, dact = z * s, s * (1 + z * (1 - s))
        e_y, e_act = 1.1 * e_z + sig * y.abs(), 0.5 * e_z + 2 * sig * (1 + z.abs())
    else:
        y, dact, e_y, e_act = z, torch.ones_like(z), e_z, torch.zeros_like(z)
    g = up * dact
    e_g = up.abs() * e_act + 2.0 ** -22 * g.abs()
    m1, m2 = mean(gm * g), mean(gm * g * xh)
    e_m1 = mean(gm.abs() * e_g) + chain * mean((gm * g).abs())
    e_m2 = mean(gm.abs() * (e_g * xh.abs() + g.abs() * e_xh)) + chain * mean((gm * g * xh).abs())
    dx = (gm * g - m1 - xh * m2) / sd
    e_dx = (gm.abs() * e_g + e_m1 + e_xh * m2.abs() + xh.abs() * e_m2) / sd + 4 * chain * (
        (gm * g).abs() + m1.abs() + (xh * m2).abs()) / sd
    dgamma, dbeta = (g * xh).sum((0, 1)), g.sum((0, 1))
    e_dg = (e_g * xh.abs() + g.abs() * e_xh).sum((0, 1)) + chain * (g * xh).abs().sum((0, 1))
    e_db = e_g.sum((0, 1)) + chain * g.abs().sum((0, 1))
    tiny = 2.0 ** -24     # fp16's smallest step
    return {"y": (y, e_y + u * (y.abs() + e_y) + tiny), "dx": (dx, e_dx + u * (dx.abs() + e_dx) + tiny),
            "dgamma": (dgamma, e_dg + pu * (dgamma.abs() + e_dg) + tiny), "dbeta": (dbeta, e_db + pu * (dbeta.abs() + e_db) + tiny)}


def run(x, dy, gamma, beta, span, act, eps=1e-5):
    y, dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device), None
    ws, stats = rf.group_norm_workspace(x, span), rf.group_norm_stats(x, span)
    rf.group_norm(x, gamma, beta, y, span=span, act=act, eps=eps, stats=stats, ws=ws)
    dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
    dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
    rf.group_norm_backward(x, gamma, beta, dy, stats, dx, dgamma, dbeta, span=span, act=act, eps=eps, ws=ws)
    return dict(y=y, dx=dx, dgamma=dgamma, dbeta=dbeta)


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_formula(name):
    x, dy, gamma, beta, span, act = make(name)
    got, want = run(x, dy, gamma, beta, span, act), reference(x, dy, gamma, beta, span, act, 1e-5)
    for nm, (value, tol) in want.items():
        off = (got[nm].double() - value).abs()
        assert (off <= tol).all(), (nm, float((off / tol).max()))


@pytest.mark.parametrize("name", ["heads_bnsd", "s_headmajor", "s_odd_width"])
def test_twice_the_same_bits(name):
    args = make(name)
    a, b = run(*args), run(*args)
    for nm in a:
        assert torch.equal(a[nm], b[nm]), nm


def test_output_strides_of_its_own():
    x, dy, gamma, beta, span, act = make("heads_bnsd")
    y = torch.empty(x.shape, dtype=x.dtype, device="cuda")        # [B, L, N, D] contiguous while x is [B, N, L, D] in memory
    rf.group_norm(x, gamma, beta, y, span=span, act=act)
    assert torch.equal(y, run(x, dy, gamma, beta, span, act)["y"])


def test_gradient_against_differences():
    """Central differences of the 64-bit loss sum(y * w) along random directions."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(2, 5, 3, 8, generator=gen).cuda()
    w = torch.randn(x.shape, generator=gen).cuda()
    gamma, beta = (1 + torch.rand(3, 8, generator=gen)).cuda(), torch.randn(3, 8, generator=gen).cuda()

    def loss(x, gamma, beta, span):
        dims = (3,) if span == "row" else (1, 3)
        mu = x.mean(dims, keepdim=True)
        z = gamma * (x - mu) / ((x - mu).pow(2).mean(dims, keepdim=True) + 1e-3).sqrt() + beta
        return (z * torch.sigmoid(z) * w.double()).sum()
    for span in ("row", "sample"):
        got = run(x, w, gamma, beta, span, "silu", eps=1e-3)
        args = [t.double() for t in (x, gamma, beta)]
        for i, nm in enumerate(("dx", "dgamma", "dbeta")):
            for _ in range(3):
                way = torch.randn(args[i].shape, generator=gen, dtype=torch.float64).cuda()
                h = 1e-5
                up, down = list(args), list(args)
                up[i], down[i] = args[i] + h * way, args[i] - h * way
                slope = float((loss(*up, span) - loss(*down, span)) / (2 * h))
                mine = float((got[nm].double() * way).sum())
                scale = float((got[nm].double() * way).abs().sum())
                # fp32 steps (2^-15 of the magnitudes) and the difference's own h^2 and rounding terms
                assert abs(slope - mine) <= 2.0 ** -15 * scale + 1e-6, (span, nm, slope, mine)


def test_empty_and_nan_stay_in_their_group():
    gamma, beta = torch.ones(2, 16, device="cuda"), torch.zeros(2, 16, device="cuda")
    x = torch.empty(0, 5, 2, 16, device="cuda")
    y, dg, db = torch.empty_like(x), torch.full_like(gamma, 7.0), torch.full_like(gamma, 7.0)
    for span in ("row", "sample"):
        rf.group_norm(x, gamma, beta, y, span=span)
        rf.group_norm_backward(x, gamma, beta, y, rf.group_norm_stats(x, span), torch.empty_like(x), dg, db, span=span)
        assert (dg == 0).all() and (db == 0).all()
    x = torch.randn(2, 70, 2, 16, device="cuda")
    x[1, 3, 0, 5] = float("nan")
    for span in ("row", "sample"):
        y = torch.empty_like(x)
        rf.group_norm(x, gamma, beta, y, span=span)
        hit = torch.zeros_like(x, dtype=torch.bool)
        if span == "row":
            hit[1, 3, 0] = True
        else:
            hit[1, :, 0] = True
        assert torch.equal(torch.isnan(y), hit)


def test_captured_and_replayed():
    x, dy, gamma, beta, span, act = make("s_odd_width")
    want = run(x, dy, gamma, beta, span, act)
    y, dx, dg, db = (torch.empty_like(t) for t in (x, x, gamma, beta))
    ws, stats = rf.group_norm_workspace(x, span), rf.group_norm_stats(x, span)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rf.group_norm(x, gamma, beta, y, span=span, act=act, stats=stats, ws=ws)
        rf.group_norm_backward(x, gamma, beta, dy, stats, dx, dg, db, span=span, act=act, ws=ws)
    for _ in range(2):
        for t in (y, dx, dg, db):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for t, nm in ((y, "y"), (dx, "dx"), (dg, "dgamma"), (db, "dbeta")):
            assert torch.equal(t, want[nm]), nm


def test_many_rows_past_32_bit_offsets():
    """A head-major view whose rows of the last head lie past 2^31 elements."""
    rows, far = 300, 2 ** 31 // 3 + 4096 - (2 ** 31 // 3) % 8
    store = torch.empty(4 * far, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((1, rows, 4, 64), (0, 64, far, 1))
    x.copy_(torch.randn(1, rows, 4, 64))
    gamma, beta = torch.ones(4, 64, device="cuda"), torch.zeros(4, 64, device="cuda")
    for span in ("row", "sample"):
        y, z = torch.empty(1, rows, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(1, rows, 4, 64, dtype=torch.bfloat16, device="cuda")
        rf.group_norm(x, gamma, beta, y, span=span)
        rf.group_norm(x.contiguous(), gamma, beta, z, span=span)
        assert torch.equal(y, z)


@pytest.mark.parametrize("span", ["row", "sample"])
def test_windows_that_share_memory(span):
    """Sliding windows over one buffer: the gradient is that of a copy of the windows, added up."""
    gen = torch.Generator().manual_seed(5)
    base = torch.randn(8 * 41, generator=gen).cuda()
    gamma, beta = (torch.randn(16, generator=gen).cuda() for _ in range(2))
    up = torch.randn(1, 40, 16, generator=gen).cuda()
    got = []
    for copied in (False, True):
        leaf = base.clone().requires_grad_()
        x = leaf.unfold(0, 16, 8)[None]
        y = diff.group_norm(x.clone(memory_format=torch.contiguous_format) if copied else x, gamma, beta, 2, span=span, act="silu")
        y.backward(up)
        got.append((y.detach(), leaf.grad))
    for a, b in zip(*got):
        assert torch.equal(a, b)
