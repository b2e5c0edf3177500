"""Differential attention in 64 bits, query block by query block, with bounds on what the kernels' roundings can change.

Rounding steps (relative, at most): the output's or gradient's own rounding u = eps / 2 of its type; P to f16 in the
forward product, 2^-11; A and dS to the tensors' type in the backward products, u.  FP32 covers the rest: scores of at
most 400 in log2 units carry an absolute error under 400 * 2^-22 there, so the exponentials are off by less than
2^-13.8, and with their sums, the products' accumulation and ex2's own 2^-22 by less than FP32 = 2^-13.

fp16 has a smallest step too: 2^-24, so a rounding there is off by 2^-25 at most whatever the value.  For the results
that is the floor itself; A carries at least 2^12 through its rounding, and dS the power of two that takes its bound
B = 2 d max|dO| max|V| max(1, |lambda|) to at most 2^15, i.e. at least 2^14 / B: their floors are smaller by that.
"""
import torch

P_STEP = 2.0 ** -11
FP32 = 2.0 ** -13
# below f16's normal range (2^-14 of the row's maximum) P has an absolute step of 2^-25 instead
P_TINY = 2.0 ** -25


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def flat(plan, x):
    """[heads, all rows, d] in 64 bits (BNSD: batch elements one behind the other)."""
    x = x.double()
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3]) if plan.layout == "BNSD" else x.transpose(0, 1)


def back(plan, x):
    return x.reshape(x.shape[0], plan.batch, -1, x.shape[2]).transpose(0, 1) if plan.layout == "BNSD" else x.transpose(0, 1)


def block_rows(plan):
    """Per sequence instance: (first global block, [(first flat row, rows) per block])."""
    out = []
    for i, s in enumerate(plan.seq_info_all()):
        base = i * int(s.length) if plan.layout == "BNSD" else int(s.row_offset)
        rows = [(base + 128 * b, min(128, int(s.lp) - 128 * b)) for b in range(s.n_pb)]
        rows += [(base + int(s.lp) + 128 * b, 128) for b in range(s.nb)]
        out.append((int(s.qblk_offset), rows))
    return out


def selection(plan, gen, keep=0.5, empty=0.0, unused=0.0):
    """Random ascending lists: each block kept with probability `keep`, whole rows emptied with probability `empty`,
    entries turned into unused slots (-1) with probability `unused`."""
    shape, shape_n = plan.select_shapes()
    idx = torch.full(shape, -1, dtype=torch.int32)
    num = torch.zeros(shape_n, dtype=torch.int32)
    for first, rows in block_rows(plan):
        n = len(rows)
        for i in range(n):
            for h in range(plan.n1):
                if torch.rand((), generator=gen) < empty:
                    continue
                pick = torch.nonzero(torch.rand(n, generator=gen) < keep).flatten().to(torch.int32)
                if len(pick) == 0 and empty == 0.0:
                    pick = torch.tensor([i], dtype=torch.int32)
                idx[first + i, h, :len(pick)] = pick
                num[first + i, h] = len(pick)
                if unused:
                    drop = torch.rand(len(pick), generator=gen) < unused
                    idx[first + i, h, :len(pick)][drop] = -1
    return idx, num


def reference(plan, q, k, v, idx, num, lam, scale, do=None):
    """{"o", "maps", "lse"} and, with do, {"dq", "dk", "dv", "dlam"}, each with a bound "<name>_tol" per element."""
    dt = q.dtype
    # an fp16 result below 2^-14 is rounded to a multiple of 2^-24 (fp16's subnormal numbers): by at most 2^-25,
    # whatever its size (bf16 has fp32's exponents and no such floor here)
    floor = 2.0 ** -25 if dt == torch.float16 else 0.0
    u, h, rep = half_step(dt), plan.d // 2, plan.n1 // plan.n2
    ds_floor = 0.0
    if do is not None and floor:
        bound = 2 * plan.d * float(do.double().abs().max()) * float(v.double().abs().max()) * max(1.0, float(lam.abs().max()))
        ds_floor = floor * bound * 2.0 ** -14
    q, k, v = (flat(plan, x) for x in (q, k, v))
    dev = q.device
    o, o_tol = torch.zeros_like(q), torch.zeros_like(q)
    maps, maps_tol = (torch.zeros(2, *q.shape, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((2, plan.n1, q.shape[1]), float("inf"), dtype=torch.float64, device=dev)
    if do is not None:
        do = flat(plan, do)
        dq, dq_tol = torch.zeros_like(q), torch.zeros_like(q)
        dk, dk_tol, dv, dv_tol = (torch.zeros_like(k) for _ in range(4))
        dlam, dlam_tol = (torch.zeros(plan.n1, dtype=torch.float64, device=dev) for _ in range(2))
    lam = lam.double().tolist()
    idx, num = idx.tolist(), num.tolist()
    for first, spans in block_rows(plan):
        rows = [torch.arange(a, a + n, device=dev) for a, n in spans]
        for i, (a, n) in enumerate(spans):
            for hd in range(plan.n1):
                pick = [j for j in idx[first + i][hd][:num[first + i][hd]] if j >= 0]
                if not pick:
                    continue
                keys, m, sl = torch.cat([rows[j] for j in pick]), hd // rep, slice(a, a + n)
                kk, vv, qq, la = k[m][keys], v[m][keys], q[hd, sl], lam[hd]
                s = [scale * (qq[:, w * h:w * h + h] @ kk[:, w * h:w * h + h].T) for w in (0, 1)]
                p = [torch.softmax(x, 1) for x in s]
                tops = [x.amax(1, keepdim=True) for x in p]      # the row maximum is 1 before division by the sum
                ow = [x @ vv for x in p]
                e = [(P_STEP + FP32) * (x @ vv.abs()) + P_TINY * t * vv.abs().sum(0) for x, t in zip(p, tops)]
                o[hd, sl] = ow[0] - la * ow[1]
                e_o = e[0] + abs(la) * e[1]
                o_tol[hd, sl] = u * (o[hd, sl].abs() + e_o) + e_o + floor
                for w in (0, 1):
                    maps[w, hd, sl], maps_tol[w, hd, sl] = ow[w], e[w]
                    lse[w, hd, sl] = torch.logsumexp(s[w], 1) / torch.log(torch.tensor(2.0, dtype=torch.float64))
                if do is None:
                    continue
                up = do[hd, sl]
                da, da_abs = up @ vv.T, up.abs() @ vv.abs().T
                big_a = p[0] - la * p[1]
                dv[m].index_add_(0, keys, big_a.T @ up)
                a_err = u * big_a.abs() + (1 + u) * FP32 * (p[0] + abs(la) * p[1])
                if dt == torch.float16:                            # A's smallest step, at the power of two it carries
                    a_err = a_err + 2.0 ** -25 * max(1.0, abs(la)) * 2.0 ** -12
                dv_tol[m].index_add_(0, keys, a_err.T @ up.abs())
                for w, c in ((0, 1.0), (1, -la)):
                    delta = (p[w] * da).sum(1, keepdim=True)
                    ds = c * p[w] * (da - delta)
                    d_err = (up.abs() * e[w]).sum(1, keepdim=True) + FP32 * (p[w] * da_abs).sum(1, keepdim=True)
                    err = u * ds.abs() + (1 + u) * abs(c) * p[w] * (d_err + FP32 * (da_abs + delta.abs())) + ds_floor
                    cols = slice(w * h, w * h + h)
                    dq[hd, sl, cols] = scale * (ds @ kk[:, cols])
                    dq_tol[hd, sl, cols] = scale * (err @ kk[:, cols].abs())
                    dk[m, :, cols].index_add_(0, keys, scale * (ds.T @ qq[:, cols]))
                    dk_tol[m, :, cols].index_add_(0, keys, scale * (err.T @ qq[:, cols].abs()))
                    if w == 1:
                        dlam[hd] -= delta.sum()
                        dlam_tol[hd] += d_err.sum()
    out = dict(o=back(plan, o), o_tol=back(plan, o_tol), maps=maps, maps_tol=maps_tol, lse=lse)
    if do is not None:
        for nm, x, t in (("dq", dq, dq_tol), ("dk", dk, dk_tol), ("dv", dv, dv_tol)):
            out[nm], out[nm + "_tol"] = back(plan, x), back(plan, t + u * (x.abs() + t) + floor)
        out["dlam"], out["dlam_tol"] = dlam, dlam_tol
    return out
