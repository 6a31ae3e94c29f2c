"""The gradients of few fp32 tokens over heads that are taken in several pieces: the pieces' hidden states' gradients
add up, labels lie in the first, an inner and the last piece, and each piece's rows of the head get theirs.

Bounds of test_gpu_head_loss, for all elements of narrow heads and on samples of wide ones. Heads of more than 2^20
rows always take several pieces; those of fewer rows here do so for their width and number of tokens.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from test_gpu_head_loss import bits, check_backward, f64, gen, matrix, scratch
from test_gpu_head_loss_large import check_sampled, forward

pytestmark = pytest.mark.gpu


def labels(n, vocab, g):
    """Ends, middle and both sides of 2^18 and 2^19 and of the pieces' usual rows; others anywhere, some outside."""
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    for i, at in enumerate((vocab - 1, 0, -1, vocab // 2, 2 ** 19, 2 ** 19 - 1, vocab, 3 * 2 ** 17, 3 * 2 ** 17 - 1, 2 ** 18)):
        if i < n and at <= vocab:
            t[i] = at
    return t


@pytest.mark.parametrize("n,vocab,dim,grad", [(1, 1100003, 9, "f32"), (7, 1200000, 16, "bf16"), (20, 1060001, 8, "f32"),
                                              (64, 1100000, 12, "f32"), (33, 2200001, 5, "bf16")])
@pytest.mark.parametrize("first", [True, False])
def test_narrow_heads(n, vocab, dim, grad, first):
    g = gen(n + dim)
    w, h = matrix(g, vocab, dim, "f32", 1, 0.3)[1], matrix(g, n, dim, "f32", 2)[1]
    t = labels(n, vocab, g)
    live = (t >= 0) & (t < vocab)
    h[~live] = float("nan")
    lse = torch.where(live, torch.logsumexp(torch.nan_to_num(h).double() @ w.double().t().contiguous(), 1), 0.0).float()
    dloss = torch.rand(n, generator=g, device="cuda") + 0.5
    dh, dw = torch.full((n, dim), float("nan"), device="cuda"), matrix(g, vocab, dim, grad, 1, 0.1)[1]
    old = dw.clone()
    big, ws = scratch(n, vocab, dim, "f32", grad)
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, dloss=dloss, scale=0.25, first=first, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all()
    check_backward(h, w, t, lse, 0.25 * f64(dloss), dh, dw, old, first)
    ws.fill_(0x5A)
    dh2, dw2 = torch.empty_like(dh), old.clone()
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh2, dw2, dloss=dloss, scale=0.25, first=first, workspace=ws)
    assert torch.equal(bits(dh2), bits(dh)) and torch.equal(bits(dw2), bits(dw))


@pytest.mark.parametrize("n,vocab,dim,grad,first", [(2, 136001, 829, "f32", True), (2, 269454, 256, "f32", False), (10, 217515, 777, "bf16", True),
                                                    (27, 1049234, 1024, "f32", True)])
def test_wide_heads(n, vocab, dim, grad, first):
    g = gen(n + dim)
    w, h = matrix(g, vocab, dim, "f32", 0, 0.05)[1], matrix(g, n, dim, "f32")[1]
    w += 0.03  # rows that do not cancel: without one piece's the hidden states' gradient is off by a tenth and more
    t = labels(n, vocab, g)
    _, lse = forward(h, w, t, "f32")
    dh, dw = torch.full((n, dim), float("nan"), device="cuda"), matrix(g, vocab, dim, grad, 0, 1e-3)[1]
    old = dw.clone()
    big, ws = scratch(n, vocab, dim, "f32", grad)
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, scale=1.0 / n, first=first, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all()
    edges = [0, 1, 81919, 81920, 114687, 114688, 196607, 196608, 524799, 524800, vocab // 2, vocab - 2, vocab - 1]
    rows = np.unique([r for r in edges if r < vocab] + [int(x) for x in t if 0 <= x < vocab])
    scale = np.float64(np.float32(1.0 / n))
    none = np.array([], np.int64)
    check_sampled(h, w, t, lse, scale, dh, dw, old, first, none, rows)
    # the hidden states' gradient against fp64 on the device, to the bound of test_gpu_head_loss without its smaller terms:
    # 2 (32 + 6 vocab / 32) 2^-24 of sum |g w|, and 2^-20 of it for the exponentials of logits within 8 of the log sum
    live = (t >= 0) & (t < vocab)
    want, size = torch.zeros(n, dim, device="cuda", dtype=torch.float64), torch.zeros(n, dim, device="cuda", dtype=torch.float64)
    for v in range(0, vocab, 1 << 16):
        wd = w[v:v + (1 << 16)].double()
        p = torch.exp(h.double() @ wd.t().contiguous() - lse.double()[:, None])
        at = (t >= v) & (t < v + len(wd))
        p[at, t[at] - v] -= 1.0
        p *= scale
        want += p @ wd
        size += p.abs() @ wd.abs()
    want[~live] = 0.0
    tol = (2 * (32 + 6 * vocab / 32) * 2.0 ** -24 + 2.0 ** -17) * size
    assert ((dh.double() - want).abs()[live] <= tol[live]).all() and (dh[~live] == 0).all()
