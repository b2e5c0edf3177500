"""Cases for timing the differential-attention operators and the group norm.

Four operators, measured through the calls that a user makes:

  attn    differential attention over the selected key blocks, for serving:
          lambda from its learned vectors, then the two softmax maps' difference
          times V.  Head n's Q and K columns [0, D/2) make the first map, columns
          [D/2, D) the second; both read the same V.
              P_w = softmax(scale * Q_w K_w^T) over the selected keys,
              O   = (P_1 - lambda P_2) V      (a row without keys gives 0)
  train   the same with its backward pass: dQ, dK, dV and the gradients of the
          four vectors lambda is made of.
  lambda  lambda_n = exp(a_n . b_n) - exp(c_n . d_n) + lambda_init, and the
          gradients of a, b, c, d.
  norm    group norm with an activation over channels-last rows, per row (each
          head on its own, after differential attention) or per sample (over all
          of its rows); with "train": its backward pass too.

Tensors of attn and train are in rearranged order (text and promoted rows first,
then whole 128-row video blocks), with the selection lists that the framework's
ranking step writes.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one rank of eight of a 40-head video layer (Wan2.2-shaped grid, ragged height)
        dict(name="attn wan 5 heads", op="attn", layout="BNSD", dtype="bf16", batch=1, seqs="512,21,30,52", n1=5, n2=5, d=128,
             sparsity=0.8, empty=False),
        # packed sequences of different geometry, grouped heads, fp16
        dict(name="attn tnd gqa", op="attn", layout="TND", dtype="fp16", batch=1, seqs="256,13,32,48;200,10,19,21", n1=8, n2=2,
             d=128, sparsity=0.8, empty=False),
        # the framework's smallest workload: two heads of 64, a few blocks
        dict(name="attn tiny", op="attn", layout="BNSD", dtype="bf16", batch=1, seqs="128,9,16,32", n1=2, n2=2, d=64, sparsity=0.8,
             empty=False),
        # text-only sequences down to a single token, packed: latency alone
        dict(name="attn single tokens", op="attn", layout="TND", dtype="bf16", batch=1,
             seqs="1,0,0,0;1,0,0,0;5,0,0,0;1,0,0,0;77,0,0,0", n1=8, n2=8, d=128, sparsity=0.8, empty=False),
        # a training step of an aligned grid, eight heads
        dict(name="train aligned 8 heads", op="train", layout="BNSD", dtype="bf16", batch=1, seqs="512,21,24,32", n1=8, n2=8, d=128,
             sparsity=0.8, empty=False),
        # packed fp16 training with grouped heads of 64, one sequence dense and ragged, rows that select nothing
        dict(name="train tnd gqa d64", op="train", layout="TND", dtype="fp16", batch=1, seqs="64,9,16,32;200,10,19,21", n1=4, n2=2,
             d=64, sparsity=0.7, empty=True),
        # lambda of one layer, per head
        dict(name="lambda layer", op="lambda", heads=40, dim=64, dtype="fp32"),
        # lambda of all layers of a model at once, 16-bit parameters
        dict(name="lambda model", op="lambda", heads=1600, dim=64, dtype="bf16"),
        # each head of the attention output on its own (BNSD: heads are the strided axis)
        dict(name="norm heads", op="norm", train=False, dtype="bf16", param="fp32", batch=1, rows=33272, groups=20, width=128,
             span="row", act="none", headmajor=True),
        # a channels-last video feature map, 32 groups, SiLU
        dict(name="norm sample silu", op="norm", train=False, dtype="bf16", param="bf16", batch=2, rows=16128, groups=32, width=10,
             span="sample", act="silu", headmajor=False),
        # training of both spans
        dict(name="norm heads train", op="norm", train=True, dtype="bf16", param="fp32", batch=1, rows=16640, groups=20, width=128,
             span="row", act="silu", headmajor=False),
        dict(name="norm sample train", op="norm", train=True, dtype="fp16", param="fp32", batch=3, rows=4567, groups=8, width=64,
             span="sample", act="silu", headmajor=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "train", "train", "lambda", "norm", "norm"])
    if op == "lambda":
        return dict(op=op, heads=_log_int(rng, 1, 1600), dim=_log_int(rng, 1, 128), dtype=rng.choice(["fp32", "bf16", "fp16"]))
    if op == "norm":
        span = rng.choice(["row", "sample"])
        return dict(op=op, train=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16", "fp32"]), param=rng.choice(["fp32", "bf16"]),
                    batch=rng.randint(1, 4), rows=_log_int(rng, 1 if span == "row" else 16, 8000), groups=rng.choice([1, 3, 8, 20, 32]),
                    width=rng.choice([8, 10, 16, 33, 64, 100, 128]), span=span, act=rng.choice(["none", "silu"]),
                    headmajor=span == "row" and rng.random() < 0.5)
    layout = rng.choice(["BNSD", "TND"])
    def video():
        while True:
            g = (rng.randint(0, 300), rng.randint(2, 16), rng.randint(8, 40), rng.randint(8, 48))
            if 700 <= g[1] * g[2] * g[3] <= 9000:
                return g
    def short():
        return (_log_int(rng, 1, 400), 0, 0, 0)
    seqs = [video()]
    if layout == "TND":
        seqs += [rng.choice([video, short])() for _ in range(rng.randint(0, 2))]
        rng.shuffle(seqs)
    elif op == "attn" and rng.random() < 0.3:
        seqs = [short()]
    n2 = rng.choice([2, 3, 4])
    return dict(op=op, layout=layout, dtype=rng.choice(["bf16", "fp16"]), batch=rng.randint(1, 2) if layout == "BNSD" else 1,
                seqs=";".join(",".join(map(str, s)) for s in seqs), n1=n2 * rng.choice([1, 2]), n2=n2, d=rng.choice([64, 128]),
                sparsity=round(rng.uniform(0.3, 0.95), 2), empty=rng.random() < 0.25)


# ---- geometry of the rearranged order -------------------------------------------------------------------

def _seqs(case):
    return [tuple(int(x) for x in s.split(",")) for s in case["seqs"].split(";")]


def _geometry(case):
    """One dict per sequence instance, in query-block order (BNSD: one per batch element)."""
    out, row, blk = [], 0, 0
    for p, t, h, w in _seqs(case) * (case["batch"] if case["layout"] == "BNSD" else 1):
        h8, w8 = h // 8 * 8, w // 8 * 8
        nb = t * h8 * w8 // 128
        length = p + t * h * w
        lp = length - 128 * nb
        npb = -(-lp // 128)
        ns = min(nb, -(-(h8 * w8) // 128))
        k = nb if nb < 32 else max(0, min(nb, math.ceil((1 - case["sparsity"]) * nb - 1e-6)))
        out.append(dict(p=p, length=length, lp=lp, nb=nb, npb=npb, ns=ns, k=k, row=row, blk=blk))
        row, blk = row + length, blk + npb + nb
    return out


def _block_rows(g):
    """First row and rows of each block of one sequence."""
    pre = [(128 * i, min(128, g["lp"] - 128 * i)) for i in range(g["npb"])]
    return pre + [(g["lp"] + 128 * i, 128) for i in range(g["nb"])]


def _selection(case, geo, gen):
    """selectIdx [blocks, n1, longest list] (ascending, padded with -1) and selectNum [blocks, n1]."""
    n1 = case["n1"]
    blocks, longest = sum(g["npb"] + g["nb"] for g in geo), max(g["npb"] + g["nb"] for g in geo)
    keep = torch.zeros(blocks, n1, longest, dtype=torch.bool, device="cuda")
    for g in geo:
        dense, n = g["npb"] + g["ns"], g["npb"] + g["nb"]
        if g["nb"] < 32:
            dense = n
        keep[g["blk"]:g["blk"] + dense, :, :n] = True
        if dense < n:
            part = keep[g["blk"] + dense:g["blk"] + n, :, :n]
            part[..., :dense] = True
            if g["k"] > 0:
                score = torch.rand(n - dense, n1, g["nb"], generator=gen, device="cuda")
                part[..., g["npb"]:].scatter_(2, score.topk(g["k"], dim=2).indices, True)
    if case["empty"]:
        keep[torch.rand(blocks, n1, generator=gen, device="cuda") < 1 / 16] = False
    at = torch.arange(longest, device="cuda").expand_as(keep)
    idx = torch.where(keep, at, longest).sort(dim=2).values
    idx = torch.where(idx == longest, -1, idx).to(torch.int32).contiguous()
    return idx, keep.sum(2, dtype=torch.int32).contiguous()


def _video(case, geo, heads, gen):
    """Text rows 0.5 N(0, 1); video rows with an offset N(0, 1) for each 64-token cell, in rearranged order."""
    n, d = heads, case["d"]
    parts = []
    for g in geo:
        x = 0.5 * torch.randn(n, g["length"], d, generator=gen, device="cuda")
        nv = g["length"] - g["p"]
        if nv:
            off = torch.randn(n, -(-nv // 64), d, generator=gen, device="cuda")
            x[:, g["length"] - nv:] += off.repeat_interleave(64, dim=1)[:, :nv]
        parts.append(x)
    dt = TYPES[case["dtype"]]
    if case["layout"] == "BNSD":
        return torch.stack(parts).to(dt).contiguous()
    return torch.cat(parts, dim=1).transpose(0, 1).to(dt).contiguous()


# ---- inputs ---------------------------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "lambda":
        dt = TYPES[case["dtype"]]
        s["vec"] = [(0.1 * torch.randn(case["heads"], case["dim"], generator=gen, device="cuda")).to(dt) for _ in range(4)]
        s["dlam"] = torch.randn(case["heads"], generator=gen, device="cuda")
        if own:
            s["lam"] = torch.empty(case["heads"], device="cuda")
            s["grad"] = [torch.empty_like(v) for v in s["vec"]]
        return s
    if case["op"] == "norm":
        dt, pt = TYPES[case["dtype"]], TYPES[case["param"]]
        shape = (case["batch"], case["rows"], case["groups"], case["width"])
        mean = torch.randn(case["groups"], case["width"], generator=gen, device="cuda")

        def rows(offset):
            x = (torch.randn(shape, generator=gen, device="cuda") + offset).to(dt)
            if case["headmajor"]:
                return x.transpose(1, 2).contiguous().transpose(1, 2)
            return x
        s["x"] = rows(mean)
        s["gamma"] = (1 + 0.1 * torch.randn(case["groups"], case["width"], generator=gen, device="cuda")).to(pt)
        s["beta"] = (0.1 * torch.randn(case["groups"], case["width"], generator=gen, device="cuda")).to(pt)
        if case["train"]:
            s["dy"] = rows(0.0)
        if own:
            from block_sparse_video_rearrange_b200 import rf
            s["y"] = torch.empty_like(s["x"])
            s["ws"] = rf.group_norm_workspace(s["x"], case["span"])
            if case["train"]:
                s["stats"] = rf.group_norm_stats(s["x"], case["span"])
                s["dx"] = torch.empty_like(s["x"])
                s["dgamma"], s["dbeta"] = torch.empty_like(s["gamma"]), torch.empty_like(s["beta"])
        return s
    geo = _geometry(case)
    dt = TYPES[case["dtype"]]
    s["geo"] = geo
    s["q"], s["k"], s["v"] = (_video(case, geo, n, gen) for n in (case["n1"], case["n2"], case["n2"]))
    s["idx"], s["num"] = _selection(case, geo, gen)
    s["vec"] = [(0.1 * torch.randn(case["n1"], case["d"] // 2, generator=gen, device="cuda")).to(dt) for _ in range(4)]
    s["scale"] = 1 / math.sqrt(case["d"] // 2)
    if case["op"] == "train":
        s["do"] = torch.randn(s["q"].shape, generator=gen, device="cuda").to(dt)
    if own:
        from block_sparse_video_rearrange_b200 import rf
        s["plan"] = rf.Plan(_seqs(case), case["n1"], case["n2"], case["d"], case["layout"], case["dtype"], case["sparsity"],
                            batch=case["batch"])
        s["bufs"] = rf.DiffBuffers(s["plan"], train=case["op"] == "train")
        s["grad"] = [torch.empty_like(v) for v in s["vec"]]
    else:
        # the block of each row of a batch element, and where the sequences' blocks begin
        per = geo[:1] if case["layout"] == "BNSD" else geo
        rows = [n for g in per for _, n in _block_rows(g)]
        s["row_block"] = torch.repeat_interleave(torch.arange(len(rows), device="cuda"), torch.tensor(rows, device="cuda"))
        s["first"] = torch.tensor([g["blk"] for g in per for _ in range(g["npb"] + g["nb"])], device="cuda")
    return s


LAMBDA_INIT = 0.8


# ---- the operators in their plain form ------------------------------------------------------------------

def _plain_lambda(vec):
    a, b, c, d = (v.float() for v in vec)
    return torch.exp((a * b).sum(-1)), torch.exp((c * d).sum(-1))


def _plain_lambda_grads(vec, e1, e2, dlam):
    a, b, c, d = (v.float() for v in vec)
    g1, g2 = (dlam * e1)[:, None], (-dlam * e2)[:, None]
    return [g.to(v.dtype) for g, v in zip((g1 * b, g1 * a, g2 * d, g2 * c), vec)]


def _plain_mask(s):
    """bool [B, n1, rows, rows]: key row selected for query row."""
    first, rb = s["first"], s["row_block"]
    idx = s["idx"].view(-1, len(first), *s["idx"].shape[1:]).long()          # [B, blocks, n1, list]
    hit = torch.zeros(*idx.shape[:3], len(first) + 1, dtype=torch.bool, device="cuda")
    hit.scatter_(3, torch.where(idx < 0, len(first), idx + first[None, :, None, None]), True)
    return hit[..., :-1].transpose(1, 2)[:, :, rb][:, :, :, rb]


def _heads_first(case, x, repeat=1):
    """[B, heads, rows, d] in fp32."""
    x = x.float() if case["layout"] == "BNSD" else x.float().transpose(0, 1)[None]
    return x.repeat_interleave(repeat, dim=1) if repeat > 1 else x


def _as_given(case, x, dtype):
    return (x if case["layout"] == "BNSD" else x[0].transpose(0, 1)).to(dtype).contiguous()


def _plain_map(q, k, mask, scale):
    s = q @ k.transpose(-1, -2)
    s = s.mul_(scale).masked_fill_(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total == 0, 1.0, total))


def _plain_attn(s):
    case, rep, h = s["case"], s["case"]["n1"] // s["case"]["n2"], s["case"]["d"] // 2
    e1, e2 = _plain_lambda(s["vec"])
    lam = (e1 - e2 + LAMBDA_INIT)[None, :, None, None]
    q, k, v = _heads_first(case, s["q"]), _heads_first(case, s["k"], rep), _heads_first(case, s["v"], rep)
    mask = _plain_mask(s)
    p1 = _plain_map(q[..., :h], k[..., :h], mask, s["scale"])
    p2 = _plain_map(q[..., h:], k[..., h:], mask, s["scale"])
    if case["op"] == "attn":
        return _as_given(case, p1.sub_(p2.mul_(lam)) @ v, s["q"].dtype)
    a = p1 - lam * p2
    o = a @ v
    do = _heads_first(case, s["do"])
    dv = a.transpose(-1, -2) @ do
    del a
    da = do @ v.transpose(-1, -2)
    t1, t2 = (p1 * da).sum(-1, keepdim=True), (p2 * da).sum(-1, keepdim=True)
    dlam = -t2.sum((0, 2, 3))
    ds1, ds2 = p1.mul_(da - t1), p2.mul_(da - t2).mul_(-lam)
    dq = s["scale"] * torch.cat([ds1 @ k[..., :h], ds2 @ k[..., h:]], -1)
    dk = s["scale"] * torch.cat([ds1.transpose(-1, -2) @ q[..., :h], ds2.transpose(-1, -2) @ q[..., h:]], -1)
    shared = (case["batch"], case["n2"], rep) if case["layout"] == "BNSD" else (1, case["n2"], rep)
    dk, dv = (x.view(*shared, *x.shape[2:]).sum(2) for x in (dk, dv))
    dt = s["q"].dtype
    return dict(o=_as_given(case, o, dt), dq=_as_given(case, dq, dt), dk=_as_given(case, dk, dt), dv=_as_given(case, dv, dt),
                dvec=_plain_lambda_grads(s["vec"], e1, e2, dlam))


def _plain_norm(s):
    case = s["case"]
    over = (3,) if case["span"] == "row" else (1, 3)
    x, gamma, beta = s["x"].float(), s["gamma"].float(), s["beta"].float()
    xc = x - x.mean(over, keepdim=True)
    rstd = torch.rsqrt((xc * xc).mean(over, keepdim=True) + 1e-5)
    xh = xc * rstd
    z = gamma * xh + beta
    silu = case["act"] == "silu"
    y = (z * torch.sigmoid(z) if silu else z).to(s["x"].dtype)
    if not case["train"]:
        return y
    dz = s["dy"].float()
    if silu:
        sg = torch.sigmoid(z)
        dz = dz * (sg * (1 + z * (1 - sg)))
    dgamma, dbeta = (dz * xh).sum((0, 1)), dz.sum((0, 1))
    g = dz * gamma
    dx = rstd * (g - g.mean(over, keepdim=True) - xh * (g * xh).mean(over, keepdim=True))
    return dict(y=y, dx=dx.to(s["x"].dtype), dgamma=dgamma.to(s["gamma"].dtype), dbeta=dbeta.to(s["beta"].dtype))


def _plain(s):
    if s["case"]["op"] == "lambda":
        e1, e2 = _plain_lambda(s["vec"])
        return dict(lam=e1 - e2 + LAMBDA_INIT, dvec=_plain_lambda_grads(s["vec"], e1, e2, s["dlam"]))
    return _plain_norm(s) if s["case"]["op"] == "norm" else _plain_attn(s)


# ---- the framework's calls ------------------------------------------------------------------------------

def _framework(s):
    from block_sparse_video_rearrange_b200 import rf
    case = s["case"]
    if case["op"] == "lambda":
        rf.diff_lambda(*s["vec"], LAMBDA_INIT, s["lam"])
        rf.diff_lambda_backward(*s["vec"], s["dlam"], *s["grad"])
        return dict(lam=s["lam"], dvec=s["grad"])
    if case["op"] == "norm":
        rf.group_norm(s["x"], s["gamma"], s["beta"], s["y"], span=case["span"], act=case["act"], eps=1e-5, stats=s.get("stats"),
                      ws=s["ws"])
        if not case["train"]:
            return s["y"]
        rf.group_norm_backward(s["x"], s["gamma"], s["beta"], s["dy"], s["stats"], s["dx"], s["dgamma"], s["dbeta"],
                               span=case["span"], act=case["act"], eps=1e-5, ws=s["ws"])
        return dict(y=s["y"], dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    b = s["bufs"]
    rf.diff_lambda(*s["vec"], LAMBDA_INIT, b.lam)
    rf.diff_attn(s["plan"], s["q"], s["k"], s["v"], s["idx"], s["num"], b.lam, s["scale"], b.o_r, b.ws, maps=b.maps, lse=b.lse)
    if case["op"] == "attn":
        return b.o_r
    rf.diff_attn_backward(s["plan"], s["q"], s["k"], s["v"], s["idx"], s["num"], b.lam, s["scale"], b.maps, b.lse, s["do"],
                          b.dq_r, b.dk_r, b.dv_r, b.dlam, b.ws)
    rf.diff_lambda_backward(*s["vec"], b.dlam, *s["grad"])
    return dict(o=b.o_r, dq=b.dq_r, dk=b.dk_r, dv=b.dv_r, dvec=s["grad"])


def run(state):
    return _framework(state) if own else _plain(state)


# ---- work -----------------------------------------------------------------------------------------------

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if case["op"] == "lambda":
        n = case["heads"] * case["dim"]
        return {"bytes": 8 * n * size + 8 * case["heads"], "flops": 12 * n}
    if case["op"] == "norm":
        n = case["batch"] * case["rows"] * case["groups"] * case["width"]
        params = case["groups"] * case["width"] * (2 if case["param"] != "fp32" else 4) * (4 if case["train"] else 2)
        return {"bytes": n * size * (4 if case["train"] else 2) + params, "flops": n * (30 if case["train"] else 10)}
    geo = _geometry(case)
    pairs = 0
    for g in geo:
        dense = g["lp"] + 128 * (g["nb"] if g["nb"] < 32 else g["ns"])
        rest = g["length"] - dense
        kept = g["ns"] + (g["k"] * (g["nb"] - g["ns"]) / g["nb"] if g["nb"] else 0)
        pairs += dense * g["length"] + rest * (g["lp"] + 128 * kept)
    pairs *= case["n1"] * (15 / 16 if case["empty"] else 1)
    rows = sum(g["length"] for g in geo)
    lists = 4 * sum(g["npb"] + g["nb"] for g in geo) * case["n1"]
    listed_blocks = pairs / case["n1"] / 128 / 128 * 4 * case["n1"]
    qo, kv = rows * case["n1"] * case["d"] * 2, rows * case["n2"] * case["d"] * 2
    if case["op"] == "attn":
        return {"bytes": 2 * qo + 2 * kv + lists + listed_blocks, "flops": 4 * case["d"] * pairs}
    return {"bytes": 4 * qo + 4 * kv + lists + listed_blocks, "flops": 12 * case["d"] * pairs}


# ---- the definitions in 64 bits -------------------------------------------------------------------------

def _exact_norm(s):
    case = s["case"]
    x = s["x"].double()
    b, r, g, w = x.shape
    gamma, beta = s["gamma"].double(), s["beta"].double()
    if case["span"] == "row":
        mu, var = x.mean(-1), x.var(-1, unbiased=False)
        mu, var = mu[..., None], var[..., None]
    else:
        flat = x.permute(0, 2, 1, 3).reshape(b, g, r * w)
        mu, var = flat.mean(-1)[:, None, :, None], flat.var(-1, unbiased=False)[:, None, :, None]
    sd = (var + 1e-5).sqrt()
    xh = (x - mu) / sd
    z = xh * gamma + beta
    y = z / (1 + torch.exp(-z)) if case["act"] == "silu" else z
    if not case["train"]:
        return y
    up = s["dy"].double()
    if case["act"] == "silu":
        sg = 1 / (1 + torch.exp(-z))
        up = up * sg + up * z * sg * (1 - sg)
    n = w if case["span"] == "row" else r * w
    dims = -1 if case["span"] == "row" else (1, 3)
    gx = up * gamma
    dx = (n * gx - gx.sum(dims, keepdim=True) - xh * (gx * xh).sum(dims, keepdim=True)) / (n * sd)
    return dict(y=y, dx=dx, dgamma=torch.einsum("brgw,brgw->gw", up, xh), dbeta=torch.einsum("brgw->gw", up))


def _exact_attn(s):
    """Query block by query block: the listed key blocks' rows gathered, everything in 64 bits."""
    case, geo, h = s["case"], s["geo"], s["case"]["d"] // 2
    bnsd, train, rep = case["layout"] == "BNSD", case["op"] == "train", case["n1"] // case["n2"]
    a, b, c, d = (v.double() for v in s["vec"])
    e1, e2 = torch.exp((a * b).sum(-1)), torch.exp((c * d).sum(-1))
    lams = (e1 - e2 + LAMBDA_INIT).tolist()

    def flat(x):       # [heads, all rows, d]: batch elements one behind the other
        return (x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3]) if bnsd else x.transpose(0, 1)).double()

    def back(x):
        return x.view(x.shape[0], case["batch"], -1, x.shape[2]).transpose(0, 1) if bnsd else x.transpose(0, 1)
    q, k, v = flat(s["q"]), flat(s["k"]), flat(s["v"])
    o = torch.zeros_like(q)
    if train:
        do, dq, dk, dv = flat(s["do"]), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dlam = torch.zeros(case["n1"], dtype=torch.float64, device="cuda")
    idx, num = s["idx"].tolist(), s["num"].tolist()
    for g in geo:
        spans = _block_rows(g)
        rows = [torch.arange(g["row"] + r0, g["row"] + r0 + n, device="cuda") for r0, n in spans]
        for i in range(len(spans)):
            r0, r1 = g["row"] + spans[i][0], g["row"] + sum(spans[i])
            for n in range(case["n1"]):
                picks = idx[g["blk"] + i][n][:num[g["blk"] + i][n]]
                if not picks:
                    continue
                keys, m = torch.cat([rows[j] for j in picks]), n // rep
                kk, vv, qq = k[m][keys], v[m][keys], q[n, r0:r1]
                p1 = torch.softmax(s["scale"] * (qq[:, :h] @ kk[:, :h].T), 1)
                p2 = torch.softmax(s["scale"] * (qq[:, h:] @ kk[:, h:].T), 1)
                o[n, r0:r1] = p1 @ vv - lams[n] * (p2 @ vv)
                if not train:
                    continue
                up = do[n, r0:r1]
                g1 = up @ vv.T
                dv[m].index_add_(0, keys, (p1 - lams[n] * p2).T @ up)
                w1, w2 = (p1 * g1).sum(1, keepdim=True), (p2 * g1).sum(1, keepdim=True)
                dlam[n] -= w2.sum()
                z1, z2 = s["scale"] * p1 * (g1 - w1), -lams[n] * s["scale"] * p2 * (g1 - w2)
                dq[n, r0:r1] = torch.cat([z1 @ kk[:, :h], z2 @ kk[:, h:]], 1)
                dk[m].index_add_(0, keys, torch.cat([z1.T @ qq[:, :h], z2.T @ qq[:, h:]], 1))
    if not train:
        return back(o)
    g1, g2 = (dlam * e1)[:, None], (-dlam * e2)[:, None]
    return dict(o=back(o), dq=back(dq), dk=back(dk), dv=back(dv), dvec=[g1 * b, g1 * a, g2 * d, g2 * c])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lambda":
        a, b, c, d = (v.double() for v in s["vec"])
        x, y = torch.exp(torch.einsum("nd,nd->n", a, b)), torch.exp(torch.einsum("nd,nd->n", c, d))
        up = s["dlam"].double()
        return dict(lam=x - y + LAMBDA_INIT, dvec=[(up * x)[:, None] * b, (up * x)[:, None] * a, -(up * y)[:, None] * d,
                                                   -(up * y)[:, None] * c])
    return _exact_norm(s) if case["op"] == "norm" else _exact_attn(s)
