"""The bounds of test_gpu_head_loss_precision see a g of fewer bits: planted in a model of the sums on the CPU.

dw[v, k] = c h with c as one, two and three bf16, added smallest first in fp32.
"""
import numpy as np
import pytest

from oracle import bf16


def to_bf16(x):
    return bf16.from_bf16_bits(bf16.to_bf16_bits(x)).astype(np.float32)


def product(c, h, planes):
    parts, left = [], c.astype(np.float32)
    for _ in range(planes):
        parts.append(to_bf16(left))
        left = (left - parts[-1]).astype(np.float32)
    s = np.zeros_like(c, np.float32)
    for p in reversed(parts):
        s = (s + p * h).astype(np.float32)  # 16 bits: the product is exact
    return s.astype(np.float64)


@pytest.mark.parametrize("planes,seen", [(1, True), (2, True), (3, False)])
def test_bits_of_g(planes, seen):
    rng = np.random.default_rng(planes)
    c = (rng.random(4000) + 0.5).astype(np.float32) * np.float32(2.0) ** rng.integers(-3, 4, 4000)
    h = to_bf16((rng.random(4000) + 0.5).astype(np.float32))
    want = c.astype(np.float64) * h.astype(np.float64)
    off = np.abs(product(c.astype(np.float32), h, planes) - want) > (3 * 2.0 ** -23 + 2 * 2.0 ** -24) * want
    assert off.mean() > 0.5 if seen else not off.any()
