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
