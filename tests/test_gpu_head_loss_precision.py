"""How many bits of g the gradients of the loss keep, element by element.

The bounds of test_gpu_head_loss add up worst cases over a whole sum, which leaves room for a g of fewer bits. Here
every sum has one term that is not zero, so that what is left is the rounding of g and of its products:

* hidden states of one nonzero column each, another one for each token, and a head of zeros: all logits are 0, and with
  log sums of 0 given, exp(z - lse) is 1: g_iv = c_i, and 0 at the label. dw[v, k] = c_i h_ik for the token i of column
  k: with g in 24 bits (three bf16) each of the three exact products is added with an error of at most a step, 2^-23 of a
  partial sum that is at most the whole: 3 2^-23, and 2^-24 for the old value's addition and 2^-24 for the last
  rounding, of |c h| + |old|. fp32 hidden states are three bf16, too: six products, and those left out are below
  2^-7 2^-16 + 2^-15 2^-8 of the whole: 2^-22 + 6 2^-23. Both are below 2^-19.8 |c h|; two bf16 keep 2^-16 at worst, and are
  further off than 2^-19.8 for most values of c.
* log sums of 200: exp(z - lse) is 0, so g is -c_i at the label and 0 elsewhere: dh_i = -c_i w_label. Of bf16
  inputs g is one bf16 and what its rounding left is added to the product: 2^-22 for the fp32 arithmetic, and half a
  step of bf16, 2^-8, for the result. Without that addition g's own 2^-8 comes on top.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from test_gpu_head_loss import DT, HALF, U, f64, gen, scratch

pytestmark = pytest.mark.gpu
# tokens and rows of the head: 256 x 64 tiles, 128 x 128 and 256 x 256 ones, sums in parts, fp32 tokens in and above the
# few that read the head in place, and above the 512 from which fp32 logits are of fp16 pairs
SIZES = [(3, 700), (40, 5000), (64, 1030), (100, 3000), (256, 60000), (300, 513), (600, 33000), (1000, 2000)]


def values(g, n):
    """c of full mantissas over some binades, none zero."""
    c = (torch.rand(n, generator=g, device="cuda") + 0.5) * torch.exp2(torch.randint(-3, 4, (n,), generator=g, device="cuda").float())
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.5, -c, c)


@pytest.mark.parametrize("n,vocab", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first", [True, False])
def test_head_gradient_in_fp32_has_24_bits_of_g(n, vocab, dtype, first):
    g = gen(n + vocab)
    dim = n + 3
    w = torch.zeros(vocab, dim, device="cuda", dtype=DT[dtype])
    at = torch.randperm(dim, generator=g, device="cuda")[:n]  # the tokens' columns
    own = values(g, n).to(DT[dtype])
    h = torch.zeros(n, dim, device="cuda", dtype=DT[dtype])
    h[torch.arange(n, device="cuda"), at] = own
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    c = values(g, n)
    dw = torch.randn(vocab, dim, generator=g, device="cuda") * 0.01
    old = dw.double()
    dh = torch.full_like(h, float("nan"))
    big, ws = scratch(n, vocab, dim, dtype, "f32")
    zs.zs_linear_cross_entropy_backward(h, w, t, torch.zeros(n, device="cuda"), dh, dw, dloss=c, first=first, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all() and (dh == 0).all()
    want = torch.zeros(vocab, dim, device="cuda", dtype=torch.float64)
    want[:, at] = (c.double() * own.double())[None, :]
    want[t, at] = 0.0
    before = torch.zeros_like(old) if first else old
    tol = (3 * 2.0 ** -23 if dtype == "bf16" else 2.0 ** -22 + 6 * 2.0 ** -23) * want.abs() + 2 * U * (want.abs() + before.abs())
    err = (dw.double() - (want + before)).abs()
    assert (err <= tol).all(), f"{(err > tol).sum().item()} off, worst {(err / tol.clamp(min=1e-300)).max().item()} of the tolerance"


@pytest.mark.parametrize("n,vocab", SIZES)
@pytest.mark.parametrize("dim", [64, 200, 777])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_hidden_gradient_in_bf16_has_the_whole_of_g_at_the_label(n, vocab, dim, grad):
    g = gen(n + vocab + dim)
    w = (torch.randn(vocab, dim, generator=g, device="cuda") * 0.1).bfloat16()
    h = torch.zeros(n, dim, device="cuda", dtype=torch.bfloat16)
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    t[: min(n, 3)] = vocab - 1
    c = values(g, n)
    dh, dw = torch.full_like(h, float("nan")), torch.empty(vocab, dim, device="cuda", dtype=DT[grad])
    big, ws = scratch(n, vocab, dim, "bf16", grad)
    zs.zs_linear_cross_entropy_backward(h, w, t, torch.full((n,), 200.0, device="cuda"), dh, dw, dloss=c, first=True, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all() and (dw == 0).all()
    want = -f64(c)[:, None] * f64(w[t])
    assert np.all(np.abs(f64(dh) - want) <= (2.0 ** -22 + HALF[torch.bfloat16]) * np.abs(want))
    # what the tolerance would say to g's bf16 alone: at least a third of the tokens' rows break it
    alone = torch.from_numpy(-f64(c.bfloat16())[:, None] * f64(w[t])).bfloat16().double().numpy()
    over = np.abs(alone - want) > (2.0 ** -22 + HALF[torch.bfloat16]) * np.abs(want)
    assert n < 40 or over.any(1).mean() > 1 / 3


@pytest.mark.parametrize("n,vocab", SIZES)
@pytest.mark.parametrize("dim", [64, 203])
@pytest.mark.parametrize("grad", ["bf16", "f32"])
def test_hidden_gradient_in_fp32_has_24_bits(n, vocab, dim, grad):
    """The same of fp32 inputs: -c w_label, of three bf16 on either side or of fp32 products."""
    g = gen(n + vocab + dim)
    w = torch.randn(vocab, dim, generator=g, device="cuda") * 0.1
    h = torch.zeros(n, dim, device="cuda")
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    t[: min(n, 3)] = vocab - 1
    c = values(g, n)
    dh, dw = torch.full_like(h, float("nan")), torch.empty(vocab, dim, device="cuda", dtype=DT[grad])
    big, ws = scratch(n, vocab, dim, "f32", grad)
    zs.zs_linear_cross_entropy_backward(h, w, t, torch.full((n,), 200.0, device="cuda"), dh, dw, dloss=c, first=True, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all() and (dw == 0).all()
    want = -f64(c)[:, None] * f64(w[t])
    assert np.all(np.abs(f64(dh) - want) <= (2.0 ** -22 + 6 * 2.0 ** -23 + U) * np.abs(want))
