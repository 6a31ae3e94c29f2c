"""The embedding's gradient where tokens' runs cross many chunks of the sorted
list: partial sums of chunks, of groups of chunks that one run covers, and
their join, for one and several tiles of columns and both types of the
gradient. Bit for bit: see _runs.py for why every right sum is exact.
"""
import pytest
import torch

import _runs
import fsdp_sharded_optimizer_flatparameter_amd as zs

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


# more than 256 chunks of 32, 64 and 128 entries, each way of sorting; up to three and five tiles of columns
@pytest.mark.parametrize("kind", list(_runs.KINDS))
@pytest.mark.parametrize("n,dim", [(9001, 5), (16384, 513), (20011, 1030), (40000, 9), (40003, 1033), (140000, 10),
                                   (140001, 523)])
@pytest.mark.parametrize("dtype,gdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
def test_sums_of_long_runs(kind, n, dim, dtype, gdt):
    t = _runs.tokens(n, kind, n).cuda()
    dout = _runs.rows(n, dim, n, "cuda")
    before = _runs.old(dim, n, "cuda")
    d = dout.to(DT[dtype])
    ws = torch.full((zs.zs_embed_workspace_bytes(n, _runs.VOCAB, dim),), 0xFF, device="cuda", dtype=torch.uint8)
    for first in (True, False):
        grad = torch.full((_runs.VOCAB, dim), float("nan"), device="cuda", dtype=DT[gdt]) if first else before.to(DT[gdt])
        zs.zs_embed_backward(d, t, grad, first=first, workspace=ws)
        want = _runs.gradient(t, dout, DT[gdt], None if first else before)
        off = bits(grad + 0.0) != bits(want + 0.0)  # a sum of zeros may keep a sign
        assert not bool(off.any()), (first, int(off.sum()), off.any(1).nonzero()[:5].tolist())
