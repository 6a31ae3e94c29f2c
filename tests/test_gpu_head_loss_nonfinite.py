"""Infinities and NaN in one token's hidden states spoil that token's loss and gradient, and no other's, in every way
that the products are made: few tokens, tiles, parts of sums, fp32 as bf16 and as fp16 planes.
"""
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from test_gpu_head_loss import DT, bits, gen, labels_of, matrix, scratch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,vocab,dim", [(6, 700, 64), (33, 700, 100), (60, 5000, 640), (64, 300, 4100), (65, 700, 64), (300, 900, 200),
                                         (600, 1030, 96), (387, 260, 2050)])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_of_hidden_states(n, vocab, dim, dtype, grad):
    g = gen(n + dim)
    w, h = matrix(g, vocab, dim, dtype, 0, dim ** -0.5)[1], matrix(g, n, dim, dtype)[1]
    t = labels_of(g, n, vocab, torch.int64, 0.0)
    spoilt = torch.zeros(n, dtype=torch.bool, device="cuda")
    spoilt[[2, 4, n - 1]] = True

    def both(hidden, lse_of=None):
        loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        _, ws = scratch(n, vocab, dim, dtype)
        zs.zs_linear_cross_entropy_forward(hidden, w, t, loss, lse=lse, workspace=ws)
        dh, dw = torch.empty_like(h), torch.empty(vocab, dim, device="cuda", dtype=DT[grad])
        _, ws = scratch(n, vocab, dim, dtype, grad)
        zs.zs_linear_cross_entropy_backward(hidden, w, t, lse if lse_of is None else lse_of, dh, dw, first=True, workspace=ws)
        return loss, lse, dh, dw

    clean = both(h)
    assert all(torch.isfinite(x).all() for x in clean)
    bad = h.clone()
    bad[2, dim - 1], bad[4, 0], bad[n - 1, dim // 2] = float("inf"), float("nan"), float("-inf")
    for lse_of in (None, clean[1]):
        loss, lse, dh, dw = both(bad, lse_of)
        assert not torch.isfinite(loss[spoilt]).any() and not torch.isfinite(dh[spoilt]).any()
        for now, was in ((loss, clean[0]), (lse, clean[1]), (dh, clean[2])):
            assert torch.equal(bits(now[~spoilt]), bits(was[~spoilt]))
    # tokens that do not count spoil nothing at all
    t[spoilt] = -100
    h[spoilt] = 1.0
    clean, out = both(h), both(bad)
    for now, was in zip(out, clean):
        assert torch.equal(bits(now), bits(was))
