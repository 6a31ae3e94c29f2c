"""What is measured of the RMS norm, the 8-bit activations and the loss.

The RMS norm with the residual's addition and its backward pass, activations
kept in 8 bits with a scale for each block of 128, and the softmax cross
entropy of a large vocabulary from the hidden states and the head's weight,
with its gradients, at the sizes of the parameter lists in synth/shapes.py
(GPT-2 small: vocabulary 50257, width 768, head tied to the embedding; the
Llama-3-8B list: 128256 x 4096; the 70B list: width 8192) and at odd ones.
Gradients of parameters go where this library takes them from: an fp32
accumulator that a micro-batch adds to (`first` false) or a contribution that
is written afresh (`first` true).

With `own` false, `run` computes the operators from elementary torch
operations in fp32; with `own` true it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "i32": 4, "i64": 8}
EPS = 1e-5
BLOCK = 128  # consecutive elements of a row that share a scale


def listed():
    return [
        # one new token of one sequence at the 70B list's width: latency
        dict(name="rms fwd 1 row 8192", op="rms_fwd", rows=1, dim=8192, dtype="bf16", stream="bf16", weight="bf16",
             residual=True, bits8=False, gap=0),
        # a micro-batch of 8 x 2048 tokens, Llama-3-8B width, the output kept in 8 bits
        dict(name="rms fwd 16k rows 4096 8 bits", op="rms_fwd", rows=16384, dim=4096, dtype="bf16", stream="bf16",
             weight="bf16", residual=True, bits8=True, gap=0),
        # the backward pass of that micro-batch: the norm's input comes from its 8-bit form, the residual's gradient
        # is added, the weight's goes into the fp32 accumulator
        dict(name="rms bwd 16k rows 4096 8 bits", op="rms_bwd", rows=16384, dim=4096, dtype="bf16", stream="bf16",
             kept="e4m3", weight="bf16", residual=True, grad="f32", first=False, gap=0),
        # odd sizes in fp32, strided rows, no residual
        dict(name="rms bwd odd sizes f32", op="rms_bwd", rows=1201, dim=1601, dtype="f32", stream="f32", kept="f32",
             weight="f32", residual=False, grad="f32", first=True, gap=5),
        # one layer's activations of a micro-batch of 8 x 2048 tokens at the 70B list's width, kept and brought back
        dict(name="pack 16k rows 8192", op="pack", rows=16384, dim=8192, dtype="bf16", gap=0),
        # odd sizes in fp32, strided rows, the last block of a row short
        dict(name="pack odd sizes f32", op="pack", rows=4999, dim=1003, dtype="f32", gap=7),
        # one token scored against the Llama-3-8B list's vocabulary: latency, and the head's weight read once
        dict(name="loss fwd 1 token Llama-8B", op="loss_fwd", n=1, vocab=128256, dim=4096, dtype="bf16", index="i64",
             ignored=0.0, gap=0),
        # a micro-batch of 8 x 1024 tokens
        dict(name="loss fwd 8k tokens Llama-8B", op="loss_fwd", n=8192, vocab=128256, dim=4096, dtype="bf16",
             index="i64", ignored=0.0, gap=0),
        # odd sizes in fp32, strided rows, a tenth of the labels ignored
        dict(name="loss fwd odd sizes f32", op="loss_fwd", n=1999, vocab=5003, dim=769, dtype="f32", index="i32",
             ignored=0.1, gap=3),
        # GPT-2 small: the head's gradient is added into the fp32 accumulator of the table that it shares
        dict(name="loss bwd GPT-2 accumulate", op="loss_bwd", n=8192, vocab=50257, dim=768, dtype="bf16", index="i64",
             grad="f32", first=False, weighted=False, ignored=0.0, gap=0),
        # a micro-batch of 8 x 1024 tokens of the Llama-3-8B list, the gradient as one bf16 contribution
        dict(name="loss bwd Llama-8B contribution", op="loss_bwd", n=8192, vocab=128256, dim=4096, dtype="bf16",
             index="i64", grad="bf16", first=True, weighted=False, ignored=0.0, gap=0),
        # odd sizes: prompts whose labels are ignored, weighted tokens, strided rows
        dict(name="loss bwd odd sizes", op="loss_bwd", n=777, vocab=9001, dim=1000, dtype="bf16", index="i32",
             grad="f32", first=True, weighted=True, ignored=0.5, gap=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: one row to 16384 (the loss: 8192), widths 64 to 8192, vocabularies of 256 to 128256, every
    type, odd sizes and strides among them."""
    op = rng.choice(["rms_fwd", "rms_bwd", "pack", "loss_fwd", "loss_bwd"])
    dim = _log(rng, 64, 8192)
    if rng.random() < 0.6:  # most widths are multiples of 64
        dim = max(64, dim // 64 * 64)
    gap = rng.choice([0, 0, 0, 1, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("loss_fwd", "loss_bwd"):
        n, vocab = _log(rng, 1, 8192), _log(rng, 256, 128256)
        while n * vocab * dim > 1 << 41:
            vocab = max(256, vocab // 2)
        case = dict(op=op, n=n, vocab=vocab, dim=dim, dtype=dtype, index=rng.choice(["i32", "i64"]),
                    ignored=rng.choice([0.0, 0.0, 0.3]) if n >= 64 else 0.0, gap=gap)
        if op == "loss_bwd":
            case.update(grad=rng.choice(["f32", "bf16"]), first=rng.random() < 0.5, weighted=rng.random() < 0.3)
        return case
    rows = _log(rng, 1, 16384)
    while rows * dim > 1 << 26:
        rows = max(1, rows // 2)
    if op == "pack":
        return dict(op=op, rows=rows, dim=dim, dtype=dtype, gap=gap)
    stream = rng.choice([dtype, "f32"])  # the residual stream's type
    case = dict(op=op, rows=rows, dim=dim, dtype=dtype, stream=stream, weight=rng.choice([dtype, "f32"]),
                residual=rng.random() < 0.7, gap=gap)
    if op == "rms_fwd":
        case.update(bits8=rng.random() < 0.4)
    else:
        case.update(kept=rng.choice([stream, "e4m3"]), grad=rng.choice(["f32", "bf16"]), first=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- inputs

def _matrix(g, rows, dim, dtype, gap, sigma, mu=0.0):
    """[rows, dim] of N(mu, sigma^2), `gap` unused elements between rows."""
    m = torch.randn(rows, dim + gap, generator=g, device="cuda", dtype=DTYPES[dtype])
    return (m.mul_(sigma).add_(mu) if mu else m.mul_(sigma))[:, :dim]


def _labels(g, c):
    """Next tokens as a text has them: frequencies fall with the rank (p ~ 1 / rank), the frequent ones lie
    scattered over the vocabulary; `ignored` of them are -100, outside of it."""
    u = torch.rand(c["n"], generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(c["vocab"] + 1.0)) - 1.0).long().clamp_(0, c["vocab"] - 1)
    t = (rank * 7919 + 13) % c["vocab"]
    if c["ignored"]:
        t[torch.rand(c["n"], generator=g, device="cuda") < c["ignored"]] = -100
    return t.to(INDEX[c["index"]])


def _hidden(g, c, weight, labels):
    """Hidden states after a norm. They lean towards their label's row, so that labels' logits are 0 to 10 higher:
    some tokens are predicted well, others not."""
    h = torch.randn(c["n"], c["dim"] + c["gap"], generator=g, device="cuda")
    lean = torch.rand(c["n"], 1, generator=g, device="cuda") * (10.0 / (c["dim"] * 4e-4))
    h[:, :c["dim"]] += lean * weight[labels.long().clamp(0, c["vocab"] - 1)].float()
    return h.to(DTYPES[c["dtype"]])[:, :c["dim"]]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] in ("loss_fwd", "loss_bwd"):
        s["weight"] = _matrix(g, c["vocab"], c["dim"], c["dtype"], c["gap"], 0.02)
        s["labels"] = _labels(g, c)
        s["hidden"] = _hidden(g, c, s["weight"], s["labels"])
        if c["op"] == "loss_fwd":
            s["loss"] = torch.empty(c["n"], device="cuda")
            s["lse"] = torch.empty(c["n"], device="cuda")
            return s
        s["lse"] = _plain_loss_fwd(s)[1]
        s["dloss"] = torch.rand(c["n"], generator=g, device="cuda") if c["weighted"] else None
        s["dhidden"] = torch.empty(c["n"], c["dim"], device="cuda", dtype=DTYPES[c["dtype"]])
        s["dweight"] = _matrix(g, c["vocab"], c["dim"], c["grad"], c["gap"], 1e-5)
        return s
    rows, dim, blocks = c["rows"], c["dim"], -(-c["dim"] // BLOCK)
    if c["op"] == "pack":
        s["x"] = _matrix(g, rows, dim, c["dtype"], c["gap"], 1.0, 0.25)
        s["codes"] = torch.empty(rows, dim, device="cuda", dtype=torch.uint8)
        s["scales"] = torch.empty(rows, blocks, device="cuda")
        s["out"] = torch.empty(rows, dim, device="cuda", dtype=DTYPES[c["dtype"]])
        return s
    s["weight"] = _matrix(g, 1, dim, c["weight"], 0, 0.1, 1.0)[0]
    if c["op"] == "rms_fwd":
        s["x"] = _matrix(g, rows, dim, c["dtype"], c["gap"], 1.0, 0.25)
        if c["residual"]:
            s["residual"] = _matrix(g, rows, dim, c["stream"], c["gap"], 3.0)
            s["sum"] = torch.empty(rows, dim, device="cuda", dtype=DTYPES[c["stream"]])
        if c["bits8"]:
            s["codes"] = torch.empty(rows, dim, device="cuda", dtype=torch.uint8)
            s["scales"] = torch.empty(rows, blocks, device="cuda")
            s["out"] = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16)
        else:
            s["y"] = torch.empty(rows, dim, device="cuda", dtype=DTYPES[c["dtype"]])
        s["rstd"] = torch.empty(rows, device="cuda")
        return s
    h = _matrix(g, rows, dim, "f32" if c["kept"] == "e4m3" else c["kept"], c["gap"], 3.0, 0.25)
    s["rstd"] = (h.float().square().mean(1) + EPS).rsqrt_()
    s["h"], s["scales"] = _plain_codes(h.float()) if c["kept"] == "e4m3" else (h, None)
    s["dy"] = _matrix(g, rows, dim, c["dtype"], c["gap"], 1e-3)
    s["dresidual"] = _matrix(g, rows, dim, c["stream"], c["gap"], 1e-3) if c["residual"] else None
    s["dh"] = torch.empty(rows, dim, device="cuda", dtype=DTYPES[c["stream"]])
    s["dweight"] = _matrix(g, 1, dim, c["grad"], 0, 1e-2)[0]
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"rms_fwd": _own_rms_fwd, "rms_bwd": _own_rms_bwd, "pack": _own_pack, "loss_fwd": _own_loss_fwd,
                "loss_bwd": _own_loss_bwd}[op](state)
    return {"rms_fwd": _plain_rms_fwd, "rms_bwd": _plain_rms_bwd, "pack": _plain_pack, "loss_fwd": _plain_loss_fwd,
            "loss_bwd": _plain_loss_bwd}[op](state)


def _own_rms_fwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    zs.zs_rms_norm_forward(s["x"], s["weight"], s.get("y"), eps=EPS, residual=s.get("residual"),
                           residual_out=s.get("sum"), codes=s.get("codes"), scales=s.get("scales"), rstd=s["rstd"])
    if s["case"]["bits8"]:
        zs.zs_activation_unpack(s["codes"], s["scales"], s["out"])
    return s.get("y"), s.get("out"), s.get("sum"), s["rstd"]


def _own_rms_bwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    c = s["case"]
    if "workspace" not in s:  # kept between passes, as a training loop keeps it
        s["workspace"] = torch.empty(zs.zs_rms_norm_workspace_bytes(c["rows"], c["dim"]), device="cuda",
                                     dtype=torch.uint8)
    zs.zs_rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dh"], scales=s["scales"],
                            dresidual=s["dresidual"], dweight=s["dweight"], first=c["first"],
                            workspace=s["workspace"])
    return s["dh"], s["dweight"]


def _own_pack(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    zs.zs_activation_pack(s["x"], s["codes"], s["scales"])
    zs.zs_activation_unpack(s["codes"], s["scales"], s["out"])
    return s["out"]


def _loss_workspace(s, grad_dtype):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    c = s["case"]
    if "workspace" not in s:
        size = zs.zs_linear_cross_entropy_workspace_bytes(c["n"], c["vocab"], c["dim"], DTYPES[c["dtype"]], grad_dtype)
        s["workspace"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    return s["workspace"]


def _own_loss_fwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    zs.zs_linear_cross_entropy_forward(s["hidden"], s["weight"], s["labels"], s["loss"], lse=s["lse"],
                                       workspace=_loss_workspace(s, None))
    return s["loss"], s["lse"]


def _own_loss_bwd(s):
    import fsdp_sharded_optimizer_flatparameter_amd as zs
    c = s["case"]
    zs.zs_linear_cross_entropy_backward(s["hidden"], s["weight"], s["labels"], s["lse"], s["dhidden"], s["dweight"],
                                        dloss=s["dloss"], scale=1.0 / c["n"], first=c["first"],
                                        workspace=_loss_workspace(s, DTYPES[c["grad"]]))
    return s["dhidden"], s["dweight"]


def _plain_codes(x):
    """e4m3 codes of fp32 rows and a scale for each block of 128: the smallest power of two with which the block's
    largest magnitude stays within 448 (1.75 * 2^8)."""
    rows, dim = x.shape
    blocks = -(-dim // BLOCK)
    padded = torch.zeros(rows, blocks * BLOCK, device=x.device)
    padded[:, :dim] = x
    padded = padded.view(rows, blocks, BLOCK)
    mantissa, exponent = torch.frexp(padded.abs().amax(2))
    exponent = exponent - 9 + (mantissa > 0.875)
    scales = torch.where(mantissa == 0, 1.0, torch.ldexp(torch.ones_like(mantissa), exponent))
    codes = (padded / scales[:, :, None]).to(torch.float8_e4m3fn)
    return codes.view(rows, blocks * BLOCK)[:, :dim].contiguous(), scales


def _plain_values(codes, scales):
    rows, dim = codes.shape
    return codes.float() * scales.repeat_interleave(BLOCK, 1)[:, :dim]


def _plain_pack(s):
    return _plain_values(*_plain_codes(s["x"].float())).to(s["x"].dtype)


def _plain_rms_fwd(s):
    h = s["x"].float()
    if "residual" in s:
        h = h + s["residual"].float()
    rstd = ((h * h).mean(1, keepdim=True) + EPS).rsqrt()
    y = h * rstd * s["weight"].float()
    total = h.to(s["residual"].dtype) if "residual" in s else None
    if s["case"]["bits8"]:
        return None, _plain_values(*_plain_codes(y)).to(torch.bfloat16), total, rstd[:, 0]
    return y.to(s["x"].dtype), None, total, rstd[:, 0]


def _plain_rms_bwd(s):
    c = s["case"]
    h = s["h"].float() if s["scales"] is None else _plain_values(s["h"], s["scales"])
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    wdy = dy * s["weight"].float()
    dh = (wdy - xhat * (wdy * xhat).mean(1, keepdim=True)) * rstd
    if c["residual"]:
        dh = dh + s["dresidual"].float()
    total = (dy * xhat).sum(0)
    s["dweight"].copy_(total if c["first"] else s["dweight"].float() + total)
    return dh.to(DTYPES[c["stream"]]), s["dweight"]


def _counted(s):
    t = s["labels"].long()
    return (t >= 0) & (t < s["case"]["vocab"]), t.clamp(0, s["case"]["vocab"] - 1)


def _plain_loss_fwd(s):
    counted, t = _counted(s)
    z = s["hidden"].float() @ s["weight"].float().t()
    top = z.amax(1, keepdim=True)
    lse = (z - top).exp_().sum(1).log_() + top[:, 0]
    loss = lse - z.gather(1, t[:, None])[:, 0]
    return torch.where(counted, loss, 0.0), torch.where(counted, lse, 0.0)


def _plain_loss_bwd(s):
    c = s["case"]
    counted, t = _counted(s)
    h, w = s["hidden"].float(), s["weight"].float()
    g = (h @ w.t()).sub_(s["lse"][:, None]).exp_()
    g[torch.arange(c["n"], device="cuda"), t] -= 1.0
    each = torch.where(counted, 1.0 / c["n"], 0.0)
    g *= (each if s["dloss"] is None else each * s["dloss"])[:, None]
    total = g.t() @ h
    s["dweight"].copy_(total if c["first"] else s["dweight"].float() + total)
    return (g @ w).to(s["hidden"].dtype), s["dweight"]


# ---------------------------------------------------------------- bytes and operations

def work(case):
    c = case
    if c["op"] in ("loss_fwd", "loss_bwd"):
        n, vocab, dim = c["n"] * (1 - c["ignored"]), c["vocab"], c["dim"]
        # the hidden states, the head's weight, the labels; a loss and a log sum for each token
        moved = (n + vocab) * dim * SIZE[c["dtype"]] + c["n"] * (SIZE[c["index"]] + 8)
        if c["op"] == "loss_fwd":
            return {"bytes": moved, "flops": 2 * n * vocab * dim}
        moved += c["n"] * dim * SIZE[c["dtype"]] + vocab * dim * SIZE[c["grad"]] * (1 if c["first"] else 2)
        # the logits again, and the two products of their gradient
        return {"bytes": moved, "flops": 6 * n * vocab * dim}
    e, r = c["rows"] * c["dim"], c["rows"]
    if c["op"] == "pack":  # read the values, write and read codes and scales, write the values
        return {"bytes": 2 * e * (SIZE[c["dtype"]] + 1) + 8 * r * -(-c["dim"] // BLOCK), "flops": 4 * e}
    moved = e * SIZE[c["dtype"]] + c["dim"] * SIZE[c["weight"]] + 4 * r
    if c["op"] == "rms_fwd":
        moved += 2 * e * SIZE[c["stream"]] if c["residual"] else 0
        # 8 bits: codes and scales are written and read, the values written
        moved += e * 4 + 8 * r * -(-c["dim"] // BLOCK) if c["bits8"] else e * SIZE[c["dtype"]]
        return {"bytes": moved, "flops": 5 * e}
    moved += e * SIZE[c["kept"]] + (4 * r * -(-c["dim"] // BLOCK) if c["kept"] == "e4m3" else 0)
    moved += e * SIZE[c["stream"]] * (2 if c["residual"] else 1)
    moved += c["dim"] * SIZE[c["grad"]] * (1 if c["first"] else 2)
    return {"bytes": moved, "flops": 10 * e}


# ---------------------------------------------------------------- the definitions in 64 bits

def _values8(x):
    """What x in fp64 stands for in 8 bits: multiples of a step of 1 / 8 of each value's power of two (of 2^-6 at
    least), in units of the block's scale; halves go to the even multiple."""
    rows, dim = x.shape
    out = torch.empty_like(x)
    for at in range(0, dim, BLOCK):
        v = x[:, at:at + BLOCK]
        top = v.abs().amax(1, keepdim=True)
        scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
        # log2 is off by a rounding where the quotient is a power of two
        scale = torch.where(top > 448.0 * scale, scale * 2.0, torch.where(top <= 224.0 * scale, scale * 0.5, scale))
        scale = torch.where(top == 0, 1.0, scale)
        q = v / scale
        step = torch.exp2(torch.frexp(q)[1].clamp(min=-5) - 4.0)
        out[:, at:at + BLOCK] = torch.round(q / step) * step * scale
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "pack":
        return _values8(s["x"].double())
    if c["op"] == "rms_fwd":
        h = s["x"].double()
        if "residual" in s:
            h += s["residual"].double()
        rstd = 1.0 / torch.sqrt(torch.linalg.vector_norm(h, dim=1).square() / c["dim"] + EPS)
        y = torch.einsum("rk,r,k->rk", h, rstd, s["weight"].double())
        total = h if "residual" in s else None
        return (None, _values8(y), total, rstd) if c["bits8"] else (y, None, total, rstd)
    if c["op"] == "rms_bwd":
        # d/dh of sum(dy * y) for y = w * h * rstd, with the statistics that the call is given
        h = s["h"].double()
        if s["scales"] is not None:
            at = torch.arange(c["dim"], device="cuda") // BLOCK
            h = h * s["scales"].double()[:, at]
        rstd, dy = s["rstd"].double(), s["dy"].double()
        inner = ((dy * h) @ s["weight"].double()) * rstd ** 3 / c["dim"]
        dh = dy * s["weight"].double() * rstd[:, None] - h * inner[:, None]
        if c["residual"]:
            dh += s["dresidual"].double()
        total = rstd @ (dy * h)
        return dh, total if c["first"] else total + s["dweight"].double()
    if c["n"] * c["vocab"] * c["dim"] > 1 << 43:
        return None
    h, t = s["hidden"].double(), s["labels"].long()
    at = torch.nonzero((t >= 0) & (t < c["vocab"]))[:, 0]
    piece = max(1, (1 << 28) // c["n"])  # rows of the head at a time
    if c["op"] == "loss_fwd":
        own_logit = (h[at] * s["weight"][t[at]].double()).sum(1)
        ratio = torch.zeros(at.numel(), device="cuda", dtype=torch.float64)  # sum of exp(z - the label's z)
        for v in range(0, c["vocab"], piece):
            ratio += torch.exp(h[at] @ s["weight"][v:v + piece].double().t() - own_logit[:, None]).sum(1)
        loss = torch.zeros(c["n"], device="cuda", dtype=torch.float64)
        lse = torch.zeros(c["n"], device="cuda", dtype=torch.float64)
        loss[at] = torch.log(ratio)
        lse[at] = loss[at] + own_logit
        return loss, lse
    each = torch.full((at.numel(),), 1.0 / c["n"], device="cuda", dtype=torch.float64)
    if s["dloss"] is not None:
        each *= s["dloss"][at].double()
    live, lse = h[at], s["lse"][at].double()
    dlive = -each[:, None] * s["weight"][t[at]].double()
    dweight = torch.zeros(c["vocab"], c["dim"], device="cuda", dtype=torch.float64)
    if not c["first"]:
        dweight += s["dweight"]
    dweight.index_add_(0, t[at], -each[:, None] * live)
    for v in range(0, c["vocab"], piece):
        w = s["weight"][v:v + piece].double()
        p = torch.exp(live @ w.t() - lse[:, None]) * each[:, None]
        dlive += p @ w
        dweight[v:v + piece] += p.t() @ live
    dhidden = torch.zeros(c["n"], c["dim"], device="cuda", dtype=torch.float64)
    dhidden[at] = dlive
    return dhidden, dweight
