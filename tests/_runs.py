"""Batches of tokens whose sorted order has long runs, with rows of small whole
numbers: every partial sum of them is exact in fp32, in any grouping, so that a
gradient has one right value and is compared bit for bit.

Rows are -3 .. 3, as many below zero as above: a sum of m of them is of the
size of 2 sqrt(m), at most 3 m < 2^24, and a part of the run that is lost or counted
twice changes it by more than the spacing of bf16 numbers of that size in
nearly every column.
"""
import torch

VOCAB = 701
# Shares of the batch in the order of the tokens' ids. What is left over is ignored.
KINDS = {
    "equal": [1.0],
    "one after many": [0.03] + [0.97],             # the first part is spread over 600 ids
    "three": [0.05, 0.41, 0.002, 0.33],            # the runs start and end within chunks
    "aligned": [8192, 8192, 1],                    # whole numbers of chunks, 64 of them too
    "off by one": [8191, 8194, 8191],
}


def tokens(n, kind, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.full((n,), -100)
    t[1::2] = VOCAB + 5
    at, parts = 0, KINDS[kind]
    for i, part in enumerate(parts):
        m = min(n - at, part if isinstance(part, int) else round(n * part))
        if len(parts) > 1 and i == 0 and not isinstance(part, int):
            t[at:at + m] = torch.randint(0, 600, (m,), generator=g)
        else:
            t[at:at + m] = VOCAB - len(parts) + i
        at += m
    return t[torch.randperm(n, generator=g)]


def rows(n, dim, seed, device="cpu"):
    g = torch.Generator(device).manual_seed(seed + 1)
    return torch.randint(-3, 4, (n, dim), generator=g, dtype=torch.int8, device=device)


def old(dim, seed, device="cpu"):
    g = torch.Generator(device).manual_seed(seed + 2)
    return torch.randint(-40, 41, (VOCAB, dim), generator=g, dtype=torch.int8, device=device)


def gradient(t, dout, dtype, before=None):
    """The sums as fp64, which holds them, rounded once to the gradient's type."""
    at = ((t >= 0) & (t < VOCAB)).nonzero()[:, 0]
    at = at[torch.argsort(t[at])]
    sums = torch.zeros(at.numel() + 1, dout.shape[1], dtype=torch.float64, device=dout.device)
    torch.cumsum(dout[at], 0, dtype=torch.float64, out=sums[1:])
    counts = torch.bincount(t[at], minlength=VOCAB)
    ends = counts.cumsum(0)
    g = sums[ends] - sums[ends - counts]
    if before is not None:
        g += before.double()
    return g.float().to(dtype)  # whole numbers below 2^24: fp32 has them as they are
