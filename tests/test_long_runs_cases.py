"""The cases of the embedding gradient's long runs tell a wrong sum from a right
one: with one chunk's part of a run lost, counted twice or taken from the
neighbour, at any of several places, the gradient differs in its bits. On the
CPU, with the mistakes planted in the reference sums."""
import pytest
import torch

import _runs


@pytest.mark.parametrize("kind", list(_runs.KINDS))
@pytest.mark.parametrize("n,dim", [(9001, 5), (40000, 9), (140000, 10)])
@pytest.mark.parametrize("chunk", [32, 64, 128])
def test_a_chunks_part_is_seen(kind, n, dim, chunk):
    t, dout, before = _runs.tokens(n, kind, n), _runs.rows(n, dim, n), _runs.old(dim, n)
    keep = ((t >= 0) & (t < _runs.VOCAB)).nonzero()[:, 0]
    order = keep[torch.sort(t[keep], stable=True).indices]
    run = t[keep].mode().values  # the longest
    at = (t[order] == run).nonzero()[:, 0]
    assert at.numel() >= 64 * chunk or n == 9001  # a run over a whole group of chunks
    first, last = int(at[0]) // chunk, int(at[-1]) // chunk
    seen = 0
    for c in {first, first + 1, (first + last) // 2, last - 1, last}:
        part = [i for i in order[c * chunk:(c + 1) * chunk].tolist() if t[i] == run]
        if not part:
            continue
        part = torch.tensor(part)
        wrong = []
        for k in (0, 2):  # lost, counted twice
            d = dout.clone()
            d[part] *= k
            wrong.append(d)
        d = dout.clone()
        nxt = order[(c + 1) * chunk:(c + 1) * chunk + part.numel()]
        if nxt.numel() == part.numel():
            d[part] = dout[nxt]  # the neighbour's
            wrong.append(d)
        for dtype in (torch.bfloat16, torch.float32):
            for old in (None, before):
                right = _runs.gradient(t, dout, dtype, old)
                for w in wrong:
                    assert not torch.equal(_runs.gradient(t, w, dtype, old), right), (c, dtype)
                    seen += 1
    assert seen >= 24


def test_every_sum_is_exact_in_fp32():
    for kind in _runs.KINDS:
        t, dout = _runs.tokens(140000, kind, 3), _runs.rows(140000, 4, 3)
        assert 3 * 140000 + 40 < 2 ** 24
        order = torch.sort(t, stable=True).indices
        sums = dout[order].float().cumsum(0)  # fp32, in order: the same as in fp64
        assert torch.equal(sums.double(), dout[order].double().cumsum(0))
