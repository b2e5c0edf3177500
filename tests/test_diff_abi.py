"""Refusals of the differential-attention and group-norm entry points: on the host, before any device call."""
import ctypes

import pytest
import torch

from block_sparse_video_rearrange_b200 import diff, rf

FAKE = [ctypes.c_void_p((i + 1) << 20) for i in range(20)]      # aligned, never dereferenced
LIB = rf.lib()


def plan(**kw):
    args = dict(seqs=[(128, 9, 16, 32)], n1=4, n2=2, d=64, layout="BNSD", dtype="bf16", sparsity=0.8)
    args.update(kw)
    return rf.Plan(**args)


def attn(p, ptr=None, scale=0.125, ws_bytes=1 << 40, **change):
    names = ["q", "k", "v", "idx", "num", "lam", "o", "maps", "lse", "ws"]
    a = dict(zip(names, FAKE))
    a.update(change)
    return LIB.rf_diff_attn(p.handle, a["q"], a["k"], a["v"], a["idx"], a["num"], a["lam"], ctypes.c_float(scale), a["o"],
                            a["maps"], a["lse"], a["ws"], ws_bytes, None)


def attn_backward(p, scale=0.125, ws_bytes=1 << 40, **change):
    names = ["q", "k", "v", "idx", "num", "lam", "maps", "lse", "do", "dq", "dk", "dv", "dlam", "ws"]
    a = dict(zip(names, FAKE))
    a.update(change)
    return LIB.rf_diff_attn_backward(p.handle, a["q"], a["k"], a["v"], a["idx"], a["num"], a["lam"], ctypes.c_float(scale),
                                     a["maps"], a["lse"], a["do"], a["dq"], a["dk"], a["dv"], a["dlam"], a["ws"], ws_bytes, None)


ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), 1), (dict(lam=None), 1), (dict(o=None), 1), (dict(ws=None), 1), (dict(idx=None), 1),
    (dict(maps=None), 1), (dict(lse=None), 1),                     # kept together or not at all
    (dict(q=ODD), 1), (dict(maps=ODD), 1), (dict(o=FAKE[0]), 1), (dict(ws=ctypes.c_void_p((9 << 20) + 16)), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(ws_bytes=16), 3),
])
def test_forward_refusals(change, status):
    assert attn(plan(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(do=None), 1), (dict(dlam=None), 1), (dict(maps=None), 1), (dict(lse=None), 1), (dict(dk=None), 1),
    (dict(dq=ODD), 1), (dict(do=ODD), 1), (dict(dq=FAKE[8]), 1), (dict(dk=FAKE[9]), 1), (dict(dv=FAKE[2]), 1),
    (dict(scale=-1.0), 1), (dict(ws_bytes=1 << 10), 3),
])
def test_backward_refusals(change, status):
    assert attn_backward(plan(), **change) == status


@pytest.mark.parametrize("kw", [dict(d=128, precision="mix"), dict(d=128, precision="fp8"), dict(precision="mxfp4"), dict(block_kv=64)])
def test_plans_it_is_not_built_for(kw):
    p = plan(**kw)
    assert attn(p) == 6 and attn_backward(p) == 6
    with pytest.raises(rf.RfError):
        rf.diff_attn_workspace_bytes(p)


def test_workspace_holds_the_plans_own():
    p = plan()
    serve, train = rf.diff_attn_workspace_bytes(p), rf.diff_attn_workspace_bytes(p, backward=True)
    blocks = int(p.info.t_qblk)
    assert p.workspace_bytes <= serve <= train
    assert serve >= p.workspace_bytes + p.n2 * blocks * 128 * p.d * 2
    assert train >= serve + p.n1 * blocks * 128 * 16


@pytest.mark.parametrize("args,status", [
    ((0, 2, 64, 4), 1), ((0, 4, 0, 4), 1), ((3, 4, 64, 4), 1), ((0, 1, 64, 0), 1),
])
def test_lambda_refusals(args, status):
    dt, rows, dim, heads = args
    assert LIB.rf_diff_lambda(*FAKE[:4], dt, rows, dim, heads, ctypes.c_float(0.8), FAKE[4], None) == status
    assert LIB.rf_diff_lambda_backward(*FAKE[:4], dt, rows, dim, heads, FAKE[4], *FAKE[5:9], None) == status


def test_lambda_refuses_null_and_infinite():
    assert LIB.rf_diff_lambda(FAKE[0], None, FAKE[2], FAKE[3], 0, 1, 8, 1, ctypes.c_float(0.8), FAKE[4], None) == 1
    assert LIB.rf_diff_lambda(*FAKE[:4], 0, 1, 8, 1, ctypes.c_float(float("inf")), FAKE[4], None) == 1
    assert LIB.rf_diff_lambda_backward(*FAKE[:4], 0, 1, 8, 1, FAKE[4], FAKE[5], None, FAKE[6], FAKE[7], None) == 1


def desc(**kw):
    d = dict(batch=2, rows=8, groups=3, width=16, x_stride_b=8 * 48, x_stride_r=48, x_stride_g=16, y_stride_b=8 * 48, y_stride_r=48,
             y_stride_g=16, dtype=0, param_dtype=2, span=1, act=1, eps=1e-5)
    d.update(kw)
    return rf.NormDesc(**d)


def norm(d, ws_bytes=1 << 40, **change):
    a = dict(zip(["x", "gamma", "beta", "y", "stats", "ws"], FAKE))
    a.update(change)
    return LIB.rf_group_norm(ctypes.byref(d), a["x"], a["gamma"], a["beta"], a["y"], a["stats"], a["ws"], ws_bytes, None)


def norm_backward(d, ws_bytes=1 << 40, **change):
    a = dict(zip(["x", "gamma", "beta", "dy", "stats", "dx", "dgamma", "dbeta", "ws"], FAKE))
    a.update(change)
    return LIB.rf_group_norm_backward(ctypes.byref(d), a["x"], a["gamma"], a["beta"], a["dy"], a["stats"], a["dx"], a["dgamma"],
                                      a["dbeta"], a["ws"], ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(groups=0), 1), (dict(width=0), 1), (dict(batch=-1), 1), (dict(dtype=3), 1), (dict(param_dtype=-1), 1), (dict(span=2), 1),
    (dict(act=7), 1), (dict(eps=-1e-5), 1), (dict(eps=float("nan")), 1), (dict(x_stride_r=-48), 1), (dict(span=0, width=1025), 6),
    (dict(rows=2 ** 31), 6), (dict(batch=70000), 6),
])
def test_norm_descriptor_refusals(kw, status):
    out = ctypes.c_int64()
    assert LIB.rf_group_norm_workspace_bytes(ctypes.byref(desc(**kw)), ctypes.byref(out)) == status
    assert norm(desc(**kw)) == status and norm_backward(desc(**kw)) == status


@pytest.mark.parametrize("kw,change", [
    ({}, dict(x=None)), ({}, dict(gamma=None)), ({}, dict(stats=None)), ({}, dict(stats=ctypes.c_void_p((5 << 20) + 4))), ({}, dict(y=FAKE[0])), ({}, dict(ws=None)),
    (dict(y_stride_b=0), {}), (dict(y_stride_r=47), {}), (dict(y_stride_g=0), {}),
])
def test_norm_call_refusals(kw, change):
    assert norm(desc(**kw), **change) == 1


@pytest.mark.parametrize("kw,change", [
    ({}, dict(dy=None)), ({}, dict(dgamma=None)), ({}, dict(stats=None)), ({}, dict(dx=FAKE[3])), (dict(x_stride_b=0), {}),
])
def test_norm_backward_refusals(kw, change):
    assert norm_backward(desc(**kw), **change) == 1


def test_norm_workspace_too_small():
    assert norm(desc(), ws_bytes=64) == 3 and norm_backward(desc(), ws_bytes=64) == 3


def test_python_refuses_host_tensors_and_wrong_shapes():
    x, g = torch.zeros(1, 4, 2, 8), torch.ones(2, 8)
    with pytest.raises(ValueError):
        rf.group_norm(x, g, g, torch.empty_like(x))
    with pytest.raises(ValueError):
        rf.group_norm(x, torch.ones(8), torch.ones(8), torch.empty_like(x))
    with pytest.raises(ValueError):
        rf.group_norm(x.transpose(2, 3), g, g, torch.empty_like(x))
    with pytest.raises(ValueError):
        diff.group_norm(x, g, g)
    with pytest.raises(ValueError):
        diff.group_norm(torch.zeros(1, 4, 10), g, g, num_groups=3)
    v = [torch.zeros(4, 8)] * 4
    with pytest.raises(ValueError):
        rf.diff_lambda(*v, 0.8, torch.empty(4))
    with pytest.raises(ValueError):
        rf.diff_lambda(*v[:3], torch.zeros(4, 9), 0.8, torch.empty(4))
    q = torch.zeros(1, 4, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        diff.rainfusion_diff_attention(q, q, q, [(128, 0, 0, 0)], v)


def test_which_layouts_share_memory():
    from block_sparse_video_rearrange_b200.diff import _overlaps
    x = torch.zeros(2, 3, 4, 8)
    assert not any(_overlaps(v) for v in (x, x.transpose(1, 2), x[:, :, 1:, :5], x[:, ::2], x[:1, :1, :1, :1], x[:, :0]))
    assert _overlaps(x[:1].expand(2, 3, 4, 8)) and _overlaps(torch.zeros(64).unfold(0, 16, 8))
