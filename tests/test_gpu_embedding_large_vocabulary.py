"""The embedding's gradient for vocabularies whose keys take three and four passes of
the sort, with marks of the touched rows of the same length, for each way of
sorting in passes. Rows are small whole numbers, so every sum is exact."""
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("vocab", [(1 << 22) - 1, 1 << 22, (1 << 27) + 1, 300_000_001])
@pytest.mark.parametrize("n", [64, 65, 1025, 16384, 32768, 32769, 70001])
def test_sums_and_zeros(vocab, n):
    g = torch.Generator(device="cuda").manual_seed(n + vocab)
    tokens = torch.randint(-vocab // 8, vocab + vocab // 8, (n,), generator=g, device="cuda")
    # repeated ones, and the same low digits under other high ones
    tokens[::3] = tokens[0].clamp(0, vocab - 1)
    some = tokens[1::3]
    some.copy_((some & 511) + (torch.arange(some.numel(), device="cuda") % 7) * (vocab // 7))
    tokens[-1], tokens[1] = vocab - 1, 0
    dout = torch.randint(-3, 4, (n, 1), generator=g, device="cuda").bfloat16()
    keep = (tokens >= 0) & (tokens < vocab)
    ids, back = torch.unique(tokens[keep], return_inverse=True)
    sums = torch.zeros(ids.numel(), device="cuda").index_add_(0, back, dout[keep, 0].float())
    ws = torch.full((zs.zs_embed_workspace_bytes(n, vocab, 1),), 0xFF, device="cuda", dtype=torch.uint8)
    grad = torch.full((vocab, 1), float("nan"), device="cuda", dtype=torch.bfloat16)
    zs.zs_embed_backward(dout, tokens, grad, first=True, workspace=ws)
    assert torch.equal(grad[ids, 0], sums.bfloat16())
    assert torch.count_nonzero(grad) == torch.count_nonzero(sums.bfloat16())  # NaN counts: all others are zeros
    grad.fill_(1.0)
    zs.zs_embed_backward(dout, tokens, grad, workspace=ws)
    assert torch.equal(grad[ids, 0], (sums + 1.0).bfloat16())
    grad[ids] = 1.0
    assert bool((grad == 1.0).all())
