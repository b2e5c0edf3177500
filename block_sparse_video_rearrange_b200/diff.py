"""Differential attention of a video layer, and the group norm that follows it.

`rainfusion_diff_attention` is the user-level call: it takes q, k, v in the
original token order, as `rf.rainfusion_attention` does, and runs the same
rearrangement, ranking and inverse around librf's differential attention

    O = (softmax(scale Q_1 K_1^T) - lambda_n softmax(scale Q_2 K_2^T)) V

per query head n over the selected blocks, Q_1, Q_2 (K_1, K_2) being the two
halves of a head's columns, with lambda made of learned vectors:
lambda_n = exp(a_n . b_n) - exp(c_n . d_n) + lambda_init.  Both calls here are
differentiable: q, k, v, the vectors, gamma and beta receive gradients (the
ranking has none, as any top-k).  The operators run in librf's kernels; torch
provides memory, streams, the autograd graph and copies: of inputs that are not
contiguous, and of a per-sequence norm's parts of a packed batch, which is one
call for each sequence.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import rf


def _refuse_capture(what: str) -> None:
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} cannot be captured into a CUDA graph: capture the calls of `rf` "
                           "(diff_attn, diff_attn_backward, group_norm, ...) with buffers of your own")


def _recording(*tensors) -> bool:
    """Whether autograd records a call on these tensors (refused inside a graph capture)."""
    train = torch.is_grad_enabled() and any(t.requires_grad for t in tensors)
    if train:
        _refuse_capture("a differentiable call")
    return train


class _DiffAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, a, b, c, d, plan, lambda_init, scale, check, train):
        dev = q.device
        bufs = rf.DiffBuffers(plan, train=train, device=dev)
        q_r, k_r, v_r = (torch.empty_like(x) for x in (q, k, v))
        si, sn = plan.select_shapes()
        idx = torch.empty(si, dtype=torch.int32, device=dev)
        num = torch.empty(sn, dtype=torch.int32, device=dev)
        o = torch.empty_like(q)
        rf.rearrange(plan, q, k, v, q_r, k_r, v_r, bufs.ws)
        rf.pool_select(plan, None, None, idx, num, bufs.ws)
        rf.diff_lambda(a, b, c, d, lambda_init, bufs.lam)
        rf.diff_attn(plan, q_r, k_r, v_r, idx, num, bufs.lam, scale, bufs.o_r, bufs.ws, maps=bufs.maps, lse=bufs.lse)
        rf.rearrange_rows(plan, bufs.o_r, o, inverse=True)
        if check:
            rf.raise_on_device_fault(plan, bufs.ws, "rainfusion_diff_attention")
        if train:
            ctx.save_for_backward(q_r, k_r, v_r, idx, num, a, b, c, d, bufs.lam, bufs.maps, bufs.lse, bufs.ws)
            ctx.plan, ctx.scale, ctx.check = plan, scale, check
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        _refuse_capture("autograd's backward pass")
        plan = ctx.plan
        q_r, k_r, v_r, idx, num, a, b, c, d, lam, maps, lse, ws = ctx.saved_tensors
        with torch.cuda.device(q_r.device):
            do_r = torch.empty_like(q_r)
            rf.rearrange_rows(plan, do.contiguous(), do_r)
            grads_r = [torch.empty_like(x) for x in (q_r, k_r, v_r)]
            dlam = torch.empty_like(lam)
            rf.diff_attn_backward(plan, q_r, k_r, v_r, idx, num, lam, ctx.scale, maps, lse, do_r, *grads_r, dlam, ws)
            grads = [torch.empty_like(x) for x in grads_r]
            for x, y in zip(grads_r, grads):
                rf.rearrange_rows(plan, x, y, inverse=True)
            vec = [torch.empty_like(x) for x in (a, b, c, d)]
            rf.diff_lambda_backward(a, b, c, d, dlam, *vec)
            if ctx.check:
                rf.raise_on_device_fault(plan, ws, "rainfusion_diff_attention (backward)")
        return (*grads, *vec, None, None, None, None, None)


def rainfusion_diff_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                              seqs: Sequence[Tuple[int, int, int, int]],
                              vectors: Sequence[torch.Tensor], lambda_init: float = 0.8, sparsity: float = 0.8,
                              layout: str = "BNSD", scale: Optional[float] = None, plan: Optional[rf.Plan] = None,
                              order: str = "tile", check: bool = True,
                              norm: Optional[Sequence[torch.Tensor]] = None, norm_span: str = "row",
                              norm_act: str = "none", eps: float = 1e-5) -> torch.Tensor:
    """Differential attention of q, k, v (original token order) on the GPU they live on.

    q, k, v, seqs, sparsity, layout and order as in `rf.rainfusion_attention`
    (device tensors, contiguous); `vectors` are lambda's four learned vectors,
    each [N1, dim], or [1, dim] shared by every head, in bf16, fp16 or fp32;
    `scale` defaults to 1 / sqrt(D / 2), each map having half a head's columns.
    A `plan` (native precision, 128 x 128 blocks) may be given instead of the
    geometry arguments.

    `norm`, when given, is (gamma, beta), each [N1, D]: the output then goes
    through `group_norm` with each head as a group, per token (norm_span "row")
    or over each sequence ("sample"), and `norm_act`.

    With check=True (the default) the forward and the backward pass synchronise
    after their kernels and raise RfError where one recorded a fault.  Inside a
    CUDA graph capture use check=False and no gradients, or the calls of `rf`.
    """
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"q must be bf16 or fp16, got {q.dtype}")
    if not q.is_cuda:
        raise ValueError("rainfusion_diff_attention takes CUDA tensors")
    if len(vectors) != 4:
        raise ValueError("lambda is made of four vectors")
    if check:
        _refuse_capture("a call with check=True")
    with torch.cuda.device(q.device):
        if plan is None:
            dtype = {torch.bfloat16: "bf16", torch.float16: "fp16"}[q.dtype]
            if layout == "BNSD":
                plan = rf.Plan(seqs, q.shape[1], k.shape[1], q.shape[3], "BNSD", dtype, sparsity, batch=q.shape[0],
                               order=order)
            else:
                plan = rf.Plan(seqs, q.shape[1], k.shape[1], q.shape[2], "TND", dtype, sparsity, order=order)
        if scale is None:
            scale = 1.0 / math.sqrt(plan.d // 2)
        q, k, v, *vectors = (x.contiguous() for x in (q, k, v, *vectors))
        o = _DiffAttention.apply(q, k, v, *vectors, plan, float(lambda_init), float(scale), check,
                                 _recording(q, k, v, *vectors))
        if norm is None:
            return o
        gamma, beta = norm
        if plan.layout == "BNSD":
            return group_norm(o.transpose(1, 2), gamma, beta, span=norm_span, act=norm_act, eps=eps).transpose(1, 2)
        if norm_span == "row" or len(plan.seqs) == 1:
            return group_norm(o[None], gamma, beta, span=norm_span, act=norm_act, eps=eps)[0]
        rows = [int(s.length) for s in plan.seq_info]
        parts = [group_norm(x[None], gamma, beta, span=norm_span, act=norm_act, eps=eps)[0] for x in o.split(rows)]
        return torch.cat(parts)


def _overlaps(x: torch.Tensor) -> bool:
    """Whether elements of x may share memory (broadcast rows, sliding windows): its gradient needs its own layout."""
    reach = 1
    for st, n in sorted((st, n) for st, n in zip(x.stride(), x.shape) if n > 1):
        if st < reach:
            return True
        reach += (n - 1) * st
    return False


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, span, act, eps, train):
        y = torch.empty_like(x)          # keeps x's strides where they are dense
        ws = rf.group_norm_workspace(x, span)
        stats = rf.group_norm_stats(x, span)
        rf.group_norm(x, gamma, beta, y, span=span, act=act, eps=eps, stats=stats, ws=ws)
        if train:
            ctx.save_for_backward(x, gamma, beta, stats, ws)
            ctx.how = (span, act, eps)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _refuse_capture("autograd's backward pass")
        x, gamma, beta, stats, ws = ctx.saved_tensors
        span, act, eps = ctx.how
        with torch.cuda.device(x.device):
            if dy.stride(3) != 1 or min(dy.stride()) < 1:      # an expanded or permuted gradient
                dy = dy.contiguous()
            dx = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=x.device)
            dgamma, dbeta = torch.empty_like(gamma), torch.empty_like(beta)
            rf.group_norm_backward(x, gamma, beta, dy, stats, dx, dgamma, dbeta, span=span, act=act, eps=eps, ws=ws)
        return dx, dgamma, dbeta, None, None, None, None


def group_norm(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, num_groups: Optional[int] = None,
               span: str = "sample", act: str = "none", eps: float = 1e-5) -> torch.Tensor:
    """Group norm with an activation of channels-last x, differentiable.

    x is [batch, rows, channels] with num_groups, or [batch, rows, groups, width]
    (any strides with contiguous channels, e.g. a BNSD tensor's transposed view);
    gamma and beta hold one value per channel ([groups, width], or flat).  Mean and
    variance are taken over a group's channels of all rows of a batch element
    (span "sample", the usual group norm) or of each row ("row").  act: "none" or
    "silu".  The result has x's shape.
    """
    shape = x.shape
    if x.dim() == 3:
        if num_groups is None or num_groups < 1 or shape[2] % num_groups:
            raise ValueError(f"{shape[2]} channels do not split into {num_groups} groups")
        x = x.unflatten(2, (num_groups, shape[2] // num_groups))
    elif x.dim() != 4:
        raise ValueError(f"x: expected [batch, rows, channels] or [batch, rows, groups, width], got {tuple(shape)}")
    elif num_groups is not None and num_groups != shape[2]:
        raise ValueError(f"num_groups is {num_groups}, but x has {shape[2]} groups")
    if not x.is_cuda:
        raise ValueError("group_norm takes CUDA tensors")
    if x.stride(3) != 1 or _overlaps(x):
        x = x.contiguous()               # rows that share memory, or channels that are not neighbours
    gw = (x.shape[2], x.shape[3])
    gamma, beta = gamma.reshape(gw).contiguous(), beta.reshape(gw).contiguous()
    with torch.cuda.device(x.device):
        y = _GroupNorm.apply(x, gamma, beta, span, act, float(eps), _recording(x, gamma, beta))
    return y.reshape(shape) if y.dim() != len(shape) else y
