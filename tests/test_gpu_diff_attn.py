"""Differential attention on a B200 against its definition in 64 bits (tests/diff_ref.py has the bounds)."""
import math

import pytest
import torch

from block_sparse_video_rearrange_b200 import rf
from tests import diff_ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# name: layout, dtype, batch, sequences (prefix, t, h, w), n1, n2, d, keep, empty rows, unused slots
CASES = {
    "one_token": ("TND", "bf16", 1, [(1, 0, 0, 0)], 1, 1, 128, 1.0, 0.0, 0.0),
    "one_token_d64": ("BNSD", "fp16", 3, [(1, 0, 0, 0)], 2, 1, 64, 1.0, 0.0, 0.0),
    "tokens_packed": ("TND", "fp16", 1, [(1, 0, 0, 0), (2, 0, 0, 0), (127, 0, 0, 0), (129, 0, 0, 0)], 2, 2, 128, 1.0, 0.0, 0.0),
    "one_block": ("BNSD", "bf16", 1, [(128, 0, 0, 0)], 1, 1, 128, 1.0, 0.0, 0.0),
    "half_block": ("BNSD", "bf16", 2, [(64, 0, 0, 0)], 2, 2, 64, 1.0, 0.0, 0.0),
    "dense_ragged": ("BNSD", "bf16", 1, [(300, 0, 0, 0)], 2, 2, 128, 1.0, 0.0, 0.0),
    "video_ragged": ("BNSD", "bf16", 1, [(77, 5, 17, 33)], 2, 2, 128, 0.6, 0.0, 0.0),
    "video_gqa": ("BNSD", "fp16", 2, [(40, 4, 16, 24)], 4, 2, 64, 0.5, 0.0, 0.2),
    "tnd_gqa_empty": ("TND", "bf16", 1, [(64, 5, 16, 24), (200, 3, 10, 19), (3, 0, 0, 0)], 6, 2, 128, 0.4, 0.3, 0.1),
    "tnd_fp16_d64": ("TND", "fp16", 1, [(0, 6, 16, 16), (130, 2, 9, 8)], 3, 3, 64, 0.5, 0.1, 0.0),
    "all_empty": ("BNSD", "bf16", 1, [(10, 2, 16, 16)], 2, 1, 128, 0.0, 1.0, 0.0),
    "many_heads": ("BNSD", "bf16", 2, [(300, 0, 0, 0)], 200, 100, 64, 0.7, 0.05, 0.0),
    "many_heads_gqa": ("TND", "fp16", 1, [(70, 3, 16, 16), (200, 0, 0, 0)], 96, 24, 128, 0.5, 0.05, 0.0),
    "many_blocks": ("BNSD", "bf16", 1, [(5, 10, 32, 32)], 1, 1, 128, 0.3, 0.0, 0.0),
}


def make(name, seed=0, spread=0.5, device="cuda"):
    layout, dtype, batch, seqs, n1, n2, d, keep, empty, unused = CASES[name]
    plan = rf.Plan(seqs, n1, n2, d, layout, dtype, 0.5, batch=batch)
    gen = torch.Generator().manual_seed(1000 + seed)
    dt = TYPES[dtype]
    q, k, v, do = (torch.randn(plan.tensor_shape(h), generator=gen) for h in (n1, n2, n2, n1))
    q, k = q * 2 * spread, k * 2 * spread
    idx, num = diff_ref.selection(plan, gen, keep, empty, unused)
    lam = 0.5 + 0.3 * torch.randn(n1, generator=gen)
    q, k, v, do = (x.to(dt).to(device) for x in (q, k, v, do))
    return plan, q, k, v, do, idx.to(device), num.to(device), lam.to(device)


def forward(plan, q, k, v, idx, num, lam, train=False, bufs=None):
    b = bufs or rf.DiffBuffers(plan, train=train)
    b.lam.copy_(lam)
    rf.diff_attn(plan, q, k, v, idx, num, b.lam, 1 / math.sqrt(plan.d // 2), b.o_r, b.ws, maps=b.maps, lse=b.lse)
    return b


def backward(plan, q, k, v, do, idx, num, b):
    rf.diff_attn_backward(plan, q, k, v, idx, num, b.lam, 1 / math.sqrt(plan.d // 2), b.maps, b.lse, do, b.dq_r, b.dk_r,
                          b.dv_r, b.dlam, b.ws)


def within(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol)
    assert not bad.any(), (what, int(bad.sum()), float((off / tol.clamp_min(1e-300)).nan_to_num(0).max()))


def ref(plan, q, k, v, idx, num, lam, do=None):
    return diff_ref.reference(plan, q, k, v, idx, num, lam, 1 / math.sqrt(plan.d // 2), do)


@pytest.mark.parametrize("name", list(CASES))
def test_forward(name):
    plan, q, k, v, do, idx, num, lam = make(name)
    b = forward(plan, q, k, v, idx, num, lam)
    want = ref(plan, q, k, v, idx, num, lam)
    within(b.o_r, want["o"], want["o_tol"], "o")
    assert rf.check_device_status(plan, b.ws) == (0, (0, 0))


@pytest.mark.parametrize("name", list(CASES))
def test_backward(name):
    plan, q, k, v, do, idx, num, lam = make(name, seed=1)
    b = forward(plan, q, k, v, idx, num, lam, train=True)
    backward(plan, q, k, v, do, idx, num, b)
    want = ref(plan, q, k, v, idx, num, lam, do)
    within(b.o_r, want["o"], want["o_tol"], "o")
    for w in (0, 1):
        within(diff_ref.flat(plan, b.maps[w]), want["maps"][w], want["maps_tol"][w], f"map {w}")
    fin = torch.isfinite(want["lse"])
    assert torch.equal(torch.isposinf(b.lse), ~fin)
    # log2 of the sum: its fp32 spacing at 64 and the relative error of the sum
    assert ((b.lse.double() - want["lse"])[fin].abs() <= 64 * 2.0 ** -22 + diff_ref.FP32).all()
    for nm, got in (("dv", b.dv_r), ("dk", b.dk_r), ("dq", b.dq_r), ("dlam", b.dlam)):
        within(got, want[nm], want[nm + "_tol"], nm)
    assert rf.check_device_status(plan, b.ws) == (0, (0, 0))


def run_all(plan, q, k, v, do, idx, num, lam, bufs=None):
    b = forward(plan, q, k, v, idx, num, lam, train=True, bufs=bufs)
    backward(plan, q, k, v, do, idx, num, b)
    return b


OUT = ("o_r", "maps", "lse", "dq_r", "dk_r", "dv_r", "dlam")


@pytest.mark.parametrize("name", ["tnd_gqa_empty", "many_heads_gqa", "video_ragged"])
def test_twice_the_same_bits(name):
    args = make(name)
    a, b = run_all(*args), run_all(*args)
    for nm in OUT:
        assert torch.equal(getattr(a, nm), getattr(b, nm)), nm


def test_serving_and_training_give_the_same_output():
    plan, q, k, v, do, idx, num, lam = make("video_gqa")
    assert torch.equal(forward(plan, q, k, v, idx, num, lam).o_r, forward(plan, q, k, v, idx, num, lam, train=True).o_r)


@pytest.mark.parametrize("spread", [0.05, 3.0])
@pytest.mark.parametrize("name", ["video_ragged", "video_gqa"])
def test_flat_and_peaked_maps(name, spread):
    """Near-uniform maps, whose difference is small beside them, and near one-hot ones, whose dS nearly cancels."""
    plan, q, k, v, do, idx, num, lam = make(name, spread=spread)
    b = run_all(plan, q, k, v, do, idx, num, lam)
    want = ref(plan, q, k, v, idx, num, lam, do)
    for nm, got in (("o", b.o_r), ("dv", b.dv_r), ("dk", b.dk_r), ("dq", b.dq_r), ("dlam", b.dlam)):
        within(got, want[nm], want[nm + "_tol"], nm)


@pytest.mark.parametrize("name,power", [("video_ragged", 40), ("video_ragged", -60), ("video_gqa", 6), ("video_gqa", -10)])
def test_v_and_its_gradient_far_from_one(name, power):
    """V in blocks of very different size: each f16 copy has its block's own power of two; fp16 gradients carry one."""
    plan, q, k, v, do, idx, num, lam = make(name)
    first = diff_ref.block_rows(plan)[0][1]
    flat = v.transpose(1, 2) if plan.layout == "BNSD" else v
    for i, (r0, n) in enumerate(first):
        if i % 2:
            flat[:, r0:r0 + n] *= 2.0 ** power
    do = do * 2.0 ** (-power if plan.dtype == "bf16" else 2)
    b = run_all(plan, q, k, v, do, idx, num, lam)
    want = ref(plan, q, k, v, idx, num, lam, do)
    # the products reach as low as fp32's normal range here: nothing below 2^-120 of it counts
    for nm, got in (("o", b.o_r), ("dv", b.dv_r), ("dk", b.dk_r), ("dq", b.dq_r)):
        within(got, want[nm], want[nm + "_tol"] + 2.0 ** (-120 if plan.dtype == "bf16" else -24), nm)


def test_large_and_negative_lambda():
    plan, q, k, v, do, idx, num, _ = make("video_gqa")
    lam = torch.tensor([-3.0, 0.0, 17.5, 1.0], device="cuda")
    b = run_all(plan, q, k, v, do, idx, num, lam)
    want = ref(plan, q, k, v, idx, num, lam, do)
    for nm, got in (("o", b.o_r), ("dv", b.dv_r), ("dk", b.dk_r), ("dq", b.dq_r), ("dlam", b.dlam)):
        within(got, want[nm], want[nm + "_tol"], nm)


def test_equal_maps_and_lambda_one_cancel():
    """Q_1 = Q_2, K_1 = K_2, lambda = 1: O is zero up to f16 rounding of P, never the size of a map."""
    plan, q, k, v, do, idx, num, lam = make("video_ragged")
    h = plan.d // 2
    q[..., h:], k[..., h:] = q[..., :h], k[..., :h]
    b = forward(plan, q, k, v, idx, num, torch.ones_like(lam))
    assert (b.o_r == 0).all()        # the two maps round alike


def test_what_lies_behind_a_block_never_counts():
    """NaN and infinity in rows that a query block does not list, and behind a sequence's last row."""
    plan, q, k, v, do, idx, num, lam = make("tnd_gqa_empty")
    clean = run_all(plan, q, k, v, do, idx, num, lam)
    first, spans = diff_ref.block_rows(plan)[1]         # the middle sequence: the others' neighbours
    rows = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
    rows[spans[0][0]:spans[-1][0] + spans[-1][1]] = True
    for bad in (float("nan"), float("inf")):
        q2, k2, v2, do2 = (x.clone() for x in (q, k, v, do))
        for x in (q2, k2, v2, do2):
            x[rows] = bad
        got = run_all(plan, q2, k2, v2, do2, idx, num, lam)
        for nm in ("o_r", "dq_r", "dk_r", "dv_r"):
            assert torch.equal(getattr(clean, nm)[~rows], getattr(got, nm)[~rows]), nm
        assert torch.equal(clean.maps[:, ~rows], got.maps[:, ~rows])


def test_entries_out_of_range_or_twice_are_skipped_and_counted():
    wide, lam = rf.Plan([(500, 0, 0, 0)], 2, 2, 128), torch.tensor([0.8, 0.3], device="cuda")
    gen = torch.Generator().manual_seed(5)
    q, k, v, do = (torch.randn(wide.tensor_shape(2), generator=gen).to(torch.bfloat16).cuda() for _ in range(4))
    good = torch.tensor([0, 1, 3, -1], dtype=torch.int32)
    messy = torch.tensor([0, 1, 1, 3], dtype=torch.int32)                       # 1 twice
    worse = torch.tensor([0, -7, 1, 3], dtype=torch.int32)                      # out of range below
    order = torch.tensor([0, 1, 3, 2], dtype=torch.int32)                       # out of order
    above = torch.tensor([0, 1, 3, 4], dtype=torch.int32)                       # no such block

    def go(row, count):
        i = row.cuda().expand(4, 2, 4).contiguous()
        n = torch.full((4, 2), count, dtype=torch.int32, device="cuda")
        b = run_all(wide, q, k, v, do, i, n, lam)
        status = rf.check_device_status(wide, b.ws)
        return b, status
    clean, status = go(good, 3)
    assert status == (0, (0, 0))
    for row in (messy, worse, order, above):
        b, status = go(row, 4)
        assert status[0] == 5 and status[1] == (2 * 8, 0)                       # both passes, every row, once each
        for nm in OUT:
            assert torch.equal(getattr(b, nm), getattr(clean, nm)), (row, nm)
    b, status = go(good, 9)                                                     # selectNum past the row: -1 unused, the count noted
    assert status[1] == (2 * 8, 0) and torch.equal(b.o_r, clean.o_r)


def test_an_expired_wait_on_record_stops_the_work():
    plan, q, k, v, do, idx, num, lam = make("one_block")
    b = rf.DiffBuffers(plan, train=True)
    rf.selftest_expired_wait(plan, b.ws)
    run_all(plan, q, k, v, do, idx, num, lam, bufs=b)
    assert (b.o_r == 0).all() and (b.dq_r == 0).all() and (b.dk_r == 0).all() and (b.dv_r == 0).all()
    with pytest.raises(rf.RfError):
        rf.raise_on_device_fault(plan, b.ws, "test")
    run_all(plan, q, k, v, do, idx, num, lam, bufs=b)
    want = ref(plan, q, k, v, idx, num, lam, do)
    within(b.dq_r, want["dq"], want["dq_tol"], "dq")


def test_captured_and_replayed_with_new_inputs():
    plan, q, k, v, do, idx, num, lam = make("video_gqa")
    b = rf.DiffBuffers(plan, train=True)
    run_all(plan, q, k, v, do, idx, num, lam, bufs=b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_all(plan, q, k, v, do, idx, num, lam, bufs=b)
    for seed in (21, 22):
        plan2, q2, k2, v2, do2, idx2, num2, lam2 = make("video_gqa", seed=seed)
        for x, y in ((q, q2), (k, k2), (v, v2), (do, do2), (idx, idx2), (num, num2), (lam, lam2)):
            x.copy_(y)
        graph.replay()
        want = run_all(plan2, q2, k2, v2, do2, idx2, num2, lam2)
        torch.cuda.synchronize()
        for nm in OUT:
            assert torch.equal(getattr(b, nm), getattr(want, nm)), nm


def test_two_streams_with_a_workspace_each():
    a_args, b_args = make("tnd_gqa_empty", seed=3), make("video_ragged", seed=4)
    want = [run_all(*a_args), run_all(*b_args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    bufs = [rf.DiffBuffers(x[0], train=True) for x in (a_args, b_args)]
    torch.cuda.synchronize()
    for _ in range(3):
        for st, args, b in zip(streams, (a_args, b_args), bufs):
            with torch.cuda.stream(st):
                run_all(*args, bufs=b)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        for nm in OUT:
            assert torch.equal(getattr(b, nm), getattr(w, nm)), nm


def test_tensors_past_32_bit_offsets():
    """Heads beyond 2^31 elements of Q and O; each row lists its own block only."""
    heads, length = 520, 33280
    plan = rf.Plan([(length, 0, 0, 0)], heads, 1, 128)
    gen = torch.Generator("cuda").manual_seed(1)
    q = torch.empty(plan.tensor_shape(heads), dtype=torch.bfloat16, device="cuda")
    for h in (0, heads - 1):
        q[0, h] = torch.randn(length, 128, generator=gen, device="cuda")
    q[0, 1:heads - 1] = q[0, 0]
    k, v = (torch.randn(plan.tensor_shape(1), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    si, sn = plan.select_shapes()
    idx = torch.full(si, -1, dtype=torch.int32, device="cuda")
    idx[..., 0] = torch.arange(si[0], device="cuda")[:, None]
    num = torch.ones(sn, dtype=torch.int32, device="cuda")
    lam = torch.full((heads,), 0.7, device="cuda")
    b = forward(plan, q, k, v, idx, num, lam)
    assert torch.equal(b.o_r[0, 0], b.o_r[0, heads // 2])
    qb, kb, vb = (x.view(-1, 128, 128).double() for x in (q[0, heads - 1], k[0, 0], v[0, 0]))
    p = [torch.softmax(qb[..., w:w + 64] @ kb[..., w:w + 64].transpose(1, 2) / 8, -1) for w in (0, 64)]
    want = (p[0] @ vb - 0.7 * (p[1] @ vb)).reshape(length, 128)
    size = ((p[0] + 0.7 * p[1]) @ vb.abs()).reshape(length, 128)
    e = (diff_ref.P_STEP + diff_ref.FP32) * size
    within(b.o_r[0, heads - 1], want, e + 2.0 ** -8 * (want.abs() + e), "o")


def test_rearrange_rows_is_the_plans_permutation():
    plan = rf.Plan([(77, 5, 17, 33)], 4, 2, 64, order="frame_pair")
    src = torch.from_numpy(plan.permutation()).cuda()
    for heads in (4, 2):
        x = torch.randn(plan.tensor_shape(heads), device="cuda").to(torch.bfloat16)
        y, z = torch.empty_like(x), torch.empty_like(x)
        rf.rearrange_rows(plan, x, y)
        assert torch.equal(y, x[:, :, src])
        rf.rearrange_rows(plan, y, z, inverse=True)
        assert torch.equal(z, x)
    with pytest.raises(rf.RfError):
        rf.rearrange_rows(plan, torch.empty(plan.tensor_shape(3), dtype=torch.bfloat16, device="cuda"),
                          torch.empty(plan.tensor_shape(3), dtype=torch.bfloat16, device="cuda"))
