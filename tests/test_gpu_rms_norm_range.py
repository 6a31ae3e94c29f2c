"""The RMS norm of rows far from one: squares that fp32 cannot hold, beside ordinary rows.

Tolerances as in test_gpu_rms_norm (u = 2^-24, d = 64 + dim / 1024): rstd to (d + 8) u, y to
(d + 12) u |y| and half a step of its type. A row whose sum of squares leaves fp32's range is
summed again times a power of two, which is exact but for elements 2^-46 of the row's largest and
smaller, whose squares are below 2^-92 of the sum: nothing beside u. Of a root mean square above
2^126 rstd is subnormal and off by another 2^-150.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import activation as oa
from oracle import rmsnorm as orn
from test_gpu_rms_norm import DT, HALF, TYPES, U, f64, gen, within

pytestmark = pytest.mark.gpu

# by kernel: 16 lanes to a row up to one wave, two waves to a row and two rows to a workgroup (bf16 2048, fp32 1024),
# a workgroup to a row, rows that are read again
DIMS = [1, 2, 7, 64, 128, 300, 768, 1024, 1031, 1536, 2048, 4096, 8192, 16384, 20001]
SIZES = [1.0, 1.1e18, 1.0, 2.0 ** 57, 1e-20, 1.0, 2.0 ** 100, 1e-37, 2.0 ** 122, 1e-25, 1.0, 2.0 ** 63, 2.0 ** -40, 1.0]


def rows_of(g, dim, dtype, sizes):
    x = torch.rand(len(sizes), dim, generator=g, device="cuda", dtype=torch.float64) + 0.5
    x *= torch.where(torch.rand(len(sizes), dim, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    return (x * torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None]).to(DT[dtype])


def check(x, r, w, eps, y, rstd, h=None, codes=None, scales=None):
    want, wh, wr = orn.rms_norm_forward(f64(x), None if w is None else f64(w), None if r is None else f64(r), eps)
    d = 64 + x.shape[1] // 1024
    tol_r = (d + 8) * U * wr + 2.0 ** -150
    within("rstd", f64(rstd), wr, tol_r)
    tol = (d + 12) * U * np.abs(want) + np.abs(wh) * (1.0 if w is None else np.abs(f64(w))) * 2.0 ** -150 + 1e-40
    within("y", f64(y), want, tol + HALF[y.dtype] * (np.abs(want) + tol))
    if h is not None:
        within("h", f64(h), wh, (U + HALF[h.dtype]) * np.abs(wh))
    if codes is not None:
        s = np.repeat(f64(scales), 128, 1)[:, :x.shape[1]]
        within("codes", oa.unpack(codes.cpu().numpy(), f64(scales)), want,
               np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * s) + tol)


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,stream", TYPES)
def test_any_size(dim, dtype, stream):
    """Rows of any size beside each other, with no eps, one that counts among the smallest, and the usual one."""
    g = gen(dim)
    for rows, eps, with_r in ((14, 0.0, False), (13, 2.0 ** -70, True), (5, float(np.float32(1e-5)), True)):
        x = rows_of(g, dim, dtype, SIZES[:rows])
        r = rows_of(g, dim, stream, [0.4 * s for s in SIZES[:rows]]) if with_r else None
        w = (torch.rand(dim, generator=g, device="cuda") + 0.5).to(DT[dtype])
        y, rstd = torch.full_like(x, float("nan")), torch.full((rows,), float("nan"), device="cuda")
        h = None if r is None else torch.empty_like(r)
        codes = torch.zeros(rows, dim, device="cuda", dtype=torch.uint8)
        scales = torch.zeros(rows, -(-dim // 128), device="cuda")
        zs.zs_rms_norm_forward(x, w, y, eps=eps, residual=r, residual_out=h, codes=codes, scales=scales, rstd=rstd)
        check(x, r, w, eps, y, rstd, h, codes, scales)
        if r is not None:  # the sum in place, the same bits
            y2, r2 = torch.empty_like(y), r.clone()
            zs.zs_rms_norm_forward(x, w, y2, eps=eps, residual=r2, residual_out=r2)
            assert torch.equal(r2, h) and torch.equal(y2, y)


@pytest.mark.parametrize("dim", [300, 2048, 8192, 20001])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_both_sides_of_the_edge(dim, dtype):
    """dim equal elements, the sum of whose squares is 2^-2, 2^0 and 2^2 times fp32's limit of 2^128 and what
    is left of its smallest step."""
    top, low = 2.0 ** 64 / dim ** 0.5, 2.0 ** -39 / dim ** 0.5
    x = torch.tensor([top * s for s in (0.5, 1.0, 2.0)] + [low * s for s in (0.5, 1.0, 2.0)] + [2.0 ** -74, 2.0 ** -75],
                     dtype=torch.float64).cuda()[:, None].expand(-1, dim).to(DT[dtype]).contiguous()
    y, rstd = torch.empty_like(x), torch.empty(len(x), device="cuda")
    zs.zs_rms_norm_forward(x, None, y, eps=0.0, rstd=rstd)
    check(x, None, None, 0.0, y, rstd)


def test_rows_that_share_a_workgroup_keep_their_bits():
    """An ordinary row's result does not depend on its neighbours' sizes."""
    for dim, dtype in ((96, "bf16"), (500, "f32"), (1000, "f32"), (2000, "bf16"), (4096, "bf16")):
        x = rows_of(gen(dim), dim, dtype, [1.0] * 40)
        y, y2 = torch.empty_like(x), torch.empty_like(x)
        zs.zs_rms_norm_forward(x, None, y)
        for size in (2.0 ** 80, 2.0 ** -80, float("inf"), float("nan")):
            far = x.clone()
            far[1::2] *= size
            zs.zs_rms_norm_forward(far, None, y2, eps=1e-5)
            assert torch.equal(y2[::2], y[::2])


@pytest.mark.parametrize("dim", [128, 4096, 20001])
def test_backward_of_the_largest(dim):
    """The statistics of such rows in the backward pass: dh is of the size of dy / |h|."""
    g = gen(dim)
    x, dy = rows_of(g, dim, "f32", [2.0 ** 70, 1.0, 2.0 ** 100]), rows_of(g, dim, "f32", [1.0, 1.0, 1.0])
    y, rstd, dh = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty_like(x)
    dw = torch.empty(dim, device="cuda")
    zs.zs_rms_norm_forward(x, None, y, rstd=rstd)
    ws = torch.empty(zs.zs_rms_norm_workspace_bytes(3, dim), device="cuda", dtype=torch.uint8)
    zs.zs_rms_norm_backward(dy, x, None, rstd, dh, dweight=dw, first=True, workspace=ws)
    want, wdw = orn.rms_norm_backward(f64(dy), f64(x), None, f64(rstd))
    xh = np.abs(f64(x)) * f64(rstd)[:, None]
    size = f64(rstd)[:, None] * (np.abs(f64(dy)) + xh * (np.abs(f64(dy)) * xh).mean(1, keepdims=True))
    within("dh", f64(dh), want, (64 + dim // 1024 + 10) * U * size + U * np.abs(want))
    within("dw", f64(dw), wdw, 10 * U * (np.abs(f64(dy)) * xh).sum(0))
