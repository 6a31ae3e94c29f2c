"""Layer norm of rows whose elements are all equal, or nearly.

By the definition the mean of equal elements is the element itself, whatever the
width and however the sum rounds: then y is the bias and rstd = 1 / sqrt(eps),
and the mean is that value. An ulp of a mean of 30000 (2^-9) times
1 / sqrt(1e-5) = 316 is 0.6 of y, so nothing less than the exact value will do.

Tolerances, u = 2^-24: rstd of a row without variance rounds eps, the root and
the quotient: 4 u. Rows that are a large value plus a small whole number of its
ulps have exact differences from that value c: what is left of the mean's error
is the rounding of the means of the row's parts and of the row itself, u |m|
each, next to that of sums of small numbers, of at most d = 64 + dim / 1024
additions, relative to what is added. With s = mean |x - c|:
|mean - m| <= 2 u |m| + (d + 2) u s = e, and y and rstd within the bounds that
general rows have for their e.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import layernorm as ol

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# one group of lanes, one wave, several waves with full and ragged ends, the walk over long rows
DIMS = [1, 2, 7, 64, 100, 127, 128, 129, 257, 448, 500, 511, 513, 769, 1031, 2056, 4095, 4104, 8200, 10240, 16391,
        20001, 33003, 40961]
VALUES = [1.0, -3.0, 0.1, 1000.0, 1000.1, -1234.567, 3.0e4, 30000.7, 1.0e6, 16777213.0]


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_equal_elements_give_the_bias(dim, dtype, wdtype):
    g = torch.Generator(device="cuda").manual_seed(dim)
    values = torch.tensor(VALUES, device="cuda").to(DT[dtype])
    x = values[:, None].expand(-1, dim).contiguous()
    w, b = (torch.randn(dim, generator=g, device="cuda").to(DT[wdtype]) for _ in range(2))
    y = torch.empty_like(x)
    mean, rstd = (torch.full((len(VALUES),), float("nan"), device="cuda") for _ in range(2))
    zs.zs_layer_norm_forward(x, w, b, y, eps=1e-5, mean=mean, rstd=rstd)
    assert torch.equal(mean, values.float()), (mean - values.float()).tolist()
    assert torch.equal(y, b.to(DT[dtype])[None].expand_as(y)), float((y.float() - b.float()).abs().max())
    assert np.all(np.abs(f64(rstd) * 1e-5 ** 0.5 - 1) <= 4 * U), rstd.tolist()


@pytest.mark.parametrize("dim", [64, 257, 500, 769, 1031, 2056, 4104, 8200, 16391, 20001, 40961])
@pytest.mark.parametrize("c", [1000.0, 30000.0, -1.0e6])
def test_small_spread_around_a_large_value(dim, c):
    g = torch.Generator(device="cuda").manual_seed(dim)
    ulp = float(np.spacing(np.float32(abs(c))))
    steps = torch.randint(-3, 4, (5, dim), generator=g, device="cuda")
    x = (c + steps.double() * ulp).float()
    assert torch.equal(x.double() - c, steps.double() * ulp)  # every element as meant
    w, b = (torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    y = torch.empty_like(x)
    mean, rstd = (torch.empty(5, device="cuda") for _ in range(2))
    zs.zs_layer_norm_forward(x, w, b, y, eps=1e-5, mean=mean, rstd=rstd)
    xd, wd, bd = f64(x), np.abs(f64(w)), np.abs(f64(b))
    want, m, r = ol.layer_norm_forward(xd, f64(w), f64(b), 1e-5)
    d = 64 + dim // 1024
    e = 2 * U * np.abs(m) + (d + 2) * U * np.abs(xd - c).mean(1)
    assert np.all(np.abs(f64(mean) - m) <= e), (f64(mean) - m) / e
    rel = (d + 8) * U + (e * r) ** 2 + 2 * U * e * r
    assert np.all(np.abs(f64(rstd) - r) <= rel * r), (f64(rstd) / r - 1) / rel
    xh = np.abs(xd - m[:, None]) * r[:, None]
    tol = wd * ((e * r)[:, None] + xh * (rel + 3 * U)[:, None]) + 2 * U * (xh * wd + bd)
    err = np.abs(f64(y) - want)
    assert np.all(err <= (tol + HALF[y.dtype] * np.abs(want)) * (1 + 2.0 ** -7)), float((err / tol).max())


@pytest.mark.parametrize("dim", [100, 768, 1031, 8200, 20001])
def test_squares_beyond_fp32(dim):
    # distances of 3e25: their squares are infinite, the sums of the elements are not, and 1 / sqrt(inf) is 0
    x = torch.full((3, dim), 3e25, device="cuda")
    x[:, 1::2] *= -1
    b = torch.randn(dim, device="cuda")
    y, rstd = torch.empty_like(x), torch.empty(3, device="cuda")
    zs.zs_layer_norm_forward(x, None, b, y, rstd=rstd)
    assert torch.count_nonzero(rstd) == 0 and torch.equal(y, b.expand_as(y))
