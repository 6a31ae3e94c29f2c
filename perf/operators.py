"""What is measured of the embedding and layer norm operators.

The embedding lookup with scaling and its gradient, and layer norm's forward
and backward pass, at the sizes of the parameter lists in synth/shapes.py
(GPT-2 small: vocabulary 50257, width 768, context 1024; the Llama-3-8B list:
128256 x 4096; the 70B list: 128256 x 8192) and at odd ones. Gradients of
parameters go where this library takes them from: an fp32 accumulator that a
micro-batch adds to (`first` false) or a contribution that is written afresh
(`first` true).

With `own` false, `run` computes the operators from elementary torch
operations in fp32; with `own` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}
EPS = 1e-5


def listed():
    return [
        # one new token of one sequence, 70B list: latency of a row copy
        dict(name="embed fwd 1 token 70B", op="embed_fwd", n=1, vocab=128256, dim=8192, pos=0, dtype="bf16",
             out="bf16", index="i64", scale=1.0, ignored=0.0, gap=0),
        # a micro-batch of 8 x 2048 tokens, Llama-3-8B list, rows scaled by sqrt(4096)
        dict(name="embed fwd 16k tokens Llama-8B", op="embed_fwd", n=16384, vocab=128256, dim=4096, pos=0,
             dtype="bf16", out="bf16", index="i64", scale=64.0, ignored=0.0, gap=0),
        # a micro-batch of 8 x 1024 tokens, GPT-2 small: token and position rows into an fp32 residual
        dict(name="embed fwd GPT-2 with positions", op="embed_fwd", n=8192, vocab=50257, dim=768, pos=1024,
             dtype="bf16", out="f32", index="i64", scale=1.0, ignored=0.0, gap=0),
        # the gradient of that micro-batch, added into the rank's fp32 accumulator
        dict(name="embed bwd GPT-2 accumulate", op="embed_bwd", n=8192, vocab=50257, dim=768, dtype="bf16",
             grad="f32", index="i64", scale=1.0, first=False, padding=-1, ignored=0.0, gap=0),
        # the whole dense gradient of the Llama-3-8B list's table as one bf16 contribution
        dict(name="embed bwd Llama-8B contribution", op="embed_bwd", n=16384, vocab=128256, dim=4096,
             dtype="bf16", grad="bf16", index="i64", scale=1.0, first=True, padding=-1, ignored=0.0, gap=0),
        # a small vocabulary (bytes and the like) at odd sizes, padding and ignored tokens, strided rows
        dict(name="embed bwd odd sizes padded", op="embed_bwd", n=4999, vocab=1003, dim=769, dtype="f32",
             grad="f32", index="i32", scale=27.75, first=True, padding=0, ignored=0.1, gap=7),
        # one new token's row at the widest hidden size: latency
        dict(name="norm fwd 1 row 8192", op="norm_fwd", rows=1, dim=8192, dtype="bf16", weight="bf16", bias=True,
             gap=0),
        # a micro-batch of 8 x 2048 rows at the 70B list's width
        dict(name="norm fwd 16k rows 8192", op="norm_fwd", rows=16384, dim=8192, dtype="bf16", weight="bf16",
             bias=True, gap=0),
        # GPT-2 small in fp32 throughout
        dict(name="norm fwd GPT-2 f32", op="norm_fwd", rows=8192, dim=768, dtype="f32", weight="f32", bias=True,
             gap=0),
        # GPT-2 small's backward, weight and bias gradients added into fp32 accumulators
        dict(name="norm bwd GPT-2 accumulate", op="norm_bwd", rows=8192, dim=768, dtype="bf16", weight="bf16",
             grad="f32", first=False, gap=0),
        # the Llama-3-8B width, gradients written as bf16 contributions
        dict(name="norm bwd 16k rows 4096", op="norm_bwd", rows=16384, dim=4096, dtype="bf16", weight="bf16",
             grad="bf16", first=True, gap=0),
        # odd sizes in fp32, strided rows
        dict(name="norm bwd odd sizes f32", op="norm_bwd", rows=1201, dim=1601, dtype="f32", weight="f32",
             grad="f32", first=True, gap=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: one row to 16384, widths 64 to 8192, every type, odd sizes and strides among them."""
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd"])
    dim = _log(rng, 64, 8192)
    if rng.random() < 0.6:  # most widths are multiples of 64
        dim = max(64, dim // 64 * 64)
    rows = _log(rng, 1, 16384)
    while rows * dim > 1 << 26:
        rows = max(1, rows // 2)
    gap = rng.choice([0, 0, 0, 1, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm_fwd":
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, weight=rng.choice([dtype, "f32"]),
                    bias=rng.random() < 0.7, gap=gap)
    if op == "norm_bwd":
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, weight=rng.choice([dtype, "f32"]),
                    grad=rng.choice(["f32", "bf16"]), first=rng.random() < 0.5, gap=gap)
    vocab = _log(rng, 256, 128256)
    while vocab * dim > 1 << 28:
        vocab = max(256, vocab // 2)
    case = dict(op=op, n=rows, vocab=vocab, dim=dim, dtype=dtype, index=rng.choice(["i32", "i64"]),
                scale=rng.choice([1.0, math.sqrt(dim)]), ignored=rng.choice([0.0, 0.0, 0.2]) if rows >= 64 else 0.0, gap=gap)
    if op == "embed_fwd":
        case.update(pos=rng.choice([0, 0, 1024]), out=rng.choice(["bf16", "f32"]))
    else:
        case.update(grad=rng.choice(["f32", "bf16"]), first=rng.random() < 0.5, padding=rng.choice([-1, -1, 0]))
    return case


# ---------------------------------------------------------------- inputs

def _matrix(g, rows, dim, dtype, gap, sigma, mu=0.0):
    """[rows, dim] of N(mu, sigma^2), `gap` unused elements between rows."""
    m = torch.randn(rows, dim + gap, generator=g, device="cuda", dtype=DTYPES[dtype])
    return (m.mul_(sigma).add_(mu) if mu else m.mul_(sigma))[:, :dim]


def _tokens(g, c):
    """Token ids as a text has them: frequencies fall with the rank (p ~ 1 / rank), the frequent ones lie
    scattered over the vocabulary; `ignored` of them are -100, outside of it."""
    u = torch.rand(c["n"], generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(c["vocab"] + 1.0)) - 1.0).long().clamp_(0, c["vocab"] - 1)
    t = (rank * 7919 + 13) % c["vocab"]
    if c["ignored"]:
        t[torch.rand(c["n"], generator=g, device="cuda") < c["ignored"]] = -100
    return t.to(INDEX[c["index"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "embed_fwd":
        s["table"] = _matrix(g, c["vocab"], c["dim"], c["dtype"], c["gap"], 0.02)
        s["tokens"] = _tokens(g, c)
        if c["pos"]:
            s["pos_table"] = _matrix(g, c["pos"], c["dim"], c["dtype"], c["gap"], 0.02)
            s["positions"] = (torch.arange(c["n"], device="cuda") % c["pos"]).to(INDEX[c["index"]])
        s["out"] = torch.empty(c["n"], c["dim"], device="cuda", dtype=DTYPES[c["out"]])
    elif c["op"] == "embed_bwd":
        s["tokens"] = _tokens(g, c)
        s["dout"] = _matrix(g, c["n"], c["dim"], c["dtype"], c["gap"], 1e-3)
        s["grad"] = _matrix(g, c["vocab"], c["dim"], c["grad"], c["gap"], 1e-3)
    else:
        s["x"] = _matrix(g, c["rows"], c["dim"], c["dtype"], c["gap"], 1.0, 0.25)
        s["weight"] = _matrix(g, 1, c["dim"], c["weight"], 0, 0.1, 1.0)[0]
        if c["op"] == "norm_fwd":
            s["bias"] = _matrix(g, 1, c["dim"], c["weight"], 0, 0.1)[0] if c["bias"] else None
            s["y"] = torch.empty(c["rows"], c["dim"], device="cuda", dtype=DTYPES[c["dtype"]])
            s["mean"] = torch.empty(c["rows"], device="cuda")
            s["rstd"] = torch.empty(c["rows"], device="cuda")
        else:
            x = s["x"].float()
            mean = x.mean(1, keepdim=True)
            s["mean"] = mean[:, 0].clone()
            s["rstd"] = ((x - mean).square_().mean(1) + EPS).rsqrt_()
            s["dy"] = _matrix(g, c["rows"], c["dim"], c["dtype"], c["gap"], 1e-3)
            s["dx"] = torch.empty(c["rows"], c["dim"], device="cuda", dtype=DTYPES[c["dtype"]])
            s["dweight"] = _matrix(g, 1, c["dim"], c["grad"], 0, 1e-2)[0]
            s["dbias"] = _matrix(g, 1, c["dim"], c["grad"], 0, 1e-2)[0]
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"embed_fwd": _own_embed_fwd, "embed_bwd": _own_embed_bwd, "norm_fwd": _own_norm_fwd,
                "norm_bwd": _own_norm_bwd}[op](state)
    return {"embed_fwd": _plain_embed_fwd, "embed_bwd": _plain_embed_bwd, "norm_fwd": _plain_norm_fwd,
            "norm_bwd": _plain_norm_bwd}[op](state)


def _own_embed_fwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    zs.zs_embed_forward(s["table"], s["tokens"], s["out"], scale=s["case"]["scale"], pos_table=s.get("pos_table"),
                        positions=s.get("positions"))
    return s["out"]


def _own_embed_bwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    c = s["case"]
    if "workspace" not in s:  # kept between passes, as a training loop keeps it
        s["workspace"] = torch.empty(zs.zs_embed_workspace_bytes(c["n"], c["vocab"], c["dim"]), device="cuda",
                                     dtype=torch.uint8)
    zs.zs_embed_backward(s["dout"], s["tokens"], s["grad"], scale=c["scale"], padding_idx=c["padding"],
                         first=c["first"], workspace=s["workspace"])
    return s["grad"]


def _own_norm_fwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    zs.zs_layer_norm_forward(s["x"], s["weight"], s["bias"], s["y"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
    return s["y"], s["mean"], s["rstd"]


def _own_norm_bwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(zs.zs_layer_norm_workspace_bytes(c["rows"], c["dim"]), device="cuda",
                                     dtype=torch.uint8)
    zs.zs_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], dweight=s["dweight"],
                              dbias=s["dbias"], first=c["first"], workspace=s["workspace"])
    return s["dx"], s["dweight"], s["dbias"]


def _lookup(table, ids):
    """fp32 rows of a table; an id outside of it gives a row of zeros."""
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[ids.clamp(0, table.shape[0] - 1)].float()
    return torch.where(inside[:, None], rows, 0.0)


def _plain_embed_fwd(s):
    c = s["case"]
    rows = _lookup(s["table"], s["tokens"]) * c["scale"]
    if c["pos"]:
        rows = rows + _lookup(s["pos_table"], s["positions"])
    return rows.to(DTYPES[c["out"]])


def _plain_embed_bwd(s):
    c, t = s["case"], s["tokens"]
    counts = (t >= 0) & (t < c["vocab"]) & (t != c["padding"])
    total = torch.zeros(c["vocab"], c["dim"], device="cuda")
    total.index_add_(0, t.clamp(0, c["vocab"] - 1), torch.where(counts[:, None], s["dout"].float(), 0.0))
    total = total * c["scale"]
    s["grad"].copy_(total if c["first"] else s["grad"].float() + total)
    return s["grad"]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = ((d * d).mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_norm_bwd(s):
    c = s["case"]
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = (s["x"].float() - s["mean"][:, None]) * rstd
    wdy = dy * s["weight"].float()
    dx = (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True)) * rstd
    for out, total in ((s["dweight"], (dy * xhat).sum(0)), (s["dbias"], dy.sum(0))):
        out.copy_(total if c["first"] else out.float() + total)
    return dx.to(s["x"].dtype), s["dweight"], s["dbias"]


# ---------------------------------------------------------------- bytes and operations

def work(case):
    c = case
    size = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
    if c["op"] == "embed_fwd":
        # the rows that the tokens select, each distinct one once, and the output
        rows = _distinct(c) + min(c["pos"], c["n"])
        moved = rows * c["dim"] * size[c["dtype"]] + c["n"] * c["dim"] * size[c["out"]]
        moved += c["n"] * size[c["index"]] * (2 if c["pos"] else 1)
        return {"bytes": moved, "flops": c["n"] * c["dim"] * (2 if c["pos"] else 1)}
    if c["op"] == "embed_bwd":
        moved = c["n"] * (1 - c["ignored"]) * c["dim"] * size[c["dtype"]] + c["n"] * size[c["index"]]
        if c["first"]:  # every row of the gradient is written
            moved += c["vocab"] * c["dim"] * size[c["grad"]]
        else:  # the rows that the tokens select are read and written
            moved += 2 * _distinct(c) * c["dim"] * size[c["grad"]]
        return {"bytes": moved, "flops": c["n"] * c["dim"]}
    e = c["rows"] * c["dim"]
    if c["op"] == "norm_fwd":
        moved = 2 * e * size[c["dtype"]] + c["dim"] * size[c["weight"]] * (2 if c["bias"] else 1) + 8 * c["rows"]
        return {"bytes": moved, "flops": 8 * e}
    moved = 3 * e * size[c["dtype"]] + c["dim"] * size[c["weight"]] + 8 * c["rows"]
    moved += 2 * c["dim"] * size[c["grad"]] * (1 if c["first"] else 2)
    return {"bytes": moved, "flops": 14 * e}


def _distinct(c):
    """Expected number of different rows that n tokens of p ~ 1 / rank select."""
    n, v = c["n"] * (1 - c["ignored"]), c["vocab"]
    total, lo = 0.0, 1.0
    while lo <= v:  # ranks in bands of a twentieth, each band taken as equally likely
        hi = min(v + 1.0, math.floor(lo * 1.05) + 1.0)
        p = math.log(hi / lo) / math.log(v + 1.0) / (hi - lo)
        total += (hi - lo) * -math.expm1(n * math.log1p(-p))
        lo = hi
    return total


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "embed_fwd":
        # zero rows stand before and behind the table for the ids outside of it
        def rows(table, ids):
            ids = ids.long()
            at = torch.where(ids < 0, -1, torch.where(ids >= table.shape[0], table.shape[0], ids)) + 1
            used, back = torch.unique(at, return_inverse=True)
            held = torch.zeros(used.numel(), table.shape[1], device="cuda", dtype=torch.float64)
            real = (used > 0) & (used <= table.shape[0])
            held[real] = table[used[real] - 1].double()
            return held[back]

        out = rows(s["table"], s["tokens"]).mul_(c["scale"])
        if c["pos"]:
            out += rows(s["pos_table"], s["positions"])
        return out
    if c["op"] == "embed_bwd":
        t = s["tokens"].long()
        at = torch.nonzero((t >= 0) & (t < c["vocab"]) & (t != c["padding"]))[:, 0]
        grad = s["grad"].double() if not c["first"] else torch.zeros(c["vocab"], c["dim"], device="cuda",
                                                                     dtype=torch.float64)
        if at.numel():
            ids, order = torch.sort(t[at], stable=True)
            run_sum = torch.cumsum(s["dout"][at[order]].double(), 0)
            last = torch.nonzero(torch.cat([ids[1:] != ids[:-1], ids.new_ones(1, dtype=torch.bool)]))[:, 0]
            ends = run_sum[last]
            grad[ids[last]] += c["scale"] * (ends - torch.cat([torch.zeros_like(ends[:1]), ends[:-1]]))
        return grad
    x = s["x"].double()
    w = s["weight"].double()
    if c["op"] == "norm_fwd":
        mean = x.sum(1) / c["dim"]
        var = (x * x).sum(1) / c["dim"] - mean * mean
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = (x * rstd[:, None] - (mean * rstd)[:, None]) * w
        return (y if s["bias"] is None else y + s["bias"].double()), mean, rstd
    # d/dx of sum(dy * y) for y = w * (x - mean) * rstd + b, with the statistics that the call is given
    rstd, dy = s["rstd"].double()[:, None], s["dy"].double()
    xhat = (x - s["mean"].double()[:, None]) * rstd
    a = dy @ w / c["dim"]
    b = (dy * xhat) @ w / c["dim"]
    dx = rstd * (dy * w - a[:, None] - xhat * b[:, None])
    old = (0.0, 0.0) if c["first"] else (s["dweight"].double(), s["dbias"].double())
    return dx, (dy * xhat).sum(0) + old[0], dy.sum(0) + old[1]
