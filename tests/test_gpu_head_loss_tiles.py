"""Whole tiles hand their results between a wave's lanes by way of LDS, ragged ones store them from registers: the
same rows of the head give the same bits either way.

A row's logits, its g and its gradient are sums over the width and over the tokens in an order that does not
depend on how many rows there are, as long as no sum is cut into parts (fewer than 16 stages of 64 values).
With the log sums given, a call over the first 100 rows alone has to repeat the first 100 rows of a call over many.
"""
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from test_gpu_head_loss import DT, bits, gen, matrix

pytestmark = pytest.mark.gpu
FEW = 100  # rows: fewer than any tile holds


@pytest.mark.parametrize("n,vocab,dim,dtype,grad", [
    # 256 x 256 tiles, then 128 x 128
    (256, 60000, 256, "bf16", "f32"), (448, 60000, 256, "bf16", "bf16"), (448, 60160, 512, "bf16", "bf16"),
    (256, 1024, 256, "bf16", "f32"), (448, 1024, 384, "bf16", "bf16"), (128, 1024, 128, "f32", "f32"),
    (128, 2048, 128, "f32", "bf16"),
])
@pytest.mark.parametrize("first", [True, False])
def test_whole_and_ragged_tiles_agree(n, vocab, dim, dtype, grad, first):
    g = gen(n + vocab)
    w, h = matrix(g, vocab, dim, dtype, 0, 0.2)[1], matrix(g, n, dim, dtype)[1]
    t = torch.randint(0, FEW, (n,), generator=g, device="cuda")
    lse = torch.rand(n, generator=g, device="cuda") * 8.0 + 4.0
    dloss = torch.randn(n, generator=g, device="cuda")
    old = matrix(g, vocab, dim, grad, 0, 0.1)[1]

    def gradient(rows):
        size = zs.zs_linear_cross_entropy_workspace_bytes(n, rows, dim, DT[dtype], DT[grad])
        ws = torch.full((size,), 0xFF, device="cuda", dtype=torch.uint8)
        dh, dw = torch.empty_like(h), old[:rows].clone()
        zs.zs_linear_cross_entropy_backward(h, w[:rows], t, lse, dh, dw, dloss=dloss, scale=0.3, first=first, workspace=ws)
        return dw

    few = gradient(FEW)
    assert torch.isfinite(few).all() and (few != 0).any(1).all()
    for _ in range(3):
        assert torch.equal(bits(gradient(vocab)[:FEW]), bits(few))
