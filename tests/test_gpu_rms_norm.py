"""The RMS norm's forward and backward pass against the fp64 oracle.

Tolerances, u = 2^-24, half = half a step of the result's type (2^-24 fp32,
2^-8 bf16), d = 64 + dim / 1024: the most additions on the way of one element in
a sum over a row (a lane adds up to 32 elements, or dim / 1024 of a row that does
not fit in registers; then come at most 6 + 16 joins).
  h:     u |h| for the addition, then half |h|
  rstd:  squares of h (2 u each) in a sum of d additions, the product with 1 / dim,
         the addition, root and quotient: relative (d + 8) u
  y:     |h rstd w| (d + 8 + 4) u + half |y|
  codes: with that y and tol: half a step of e4m3, 2^-4 |y| or 2^-10 scales, and tol; the scale is
         that of a largest magnitude within tol of the exact one
  dh:    S = rstd (|g| + |xh| mean |g xh|) for g = dy w, statistics as given: (d + 8) u S
         + 2 u (S + |dres|) + half |dh|
  dw:    (rows + 6) u (|old| + sum |dy xh|) + half |dw|
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import activation as oa
from oracle import rmsnorm as orn

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DIMS = [1, 2, 7, 64, 127, 128, 129, 257, 512, 513, 768, 1024, 1031, 1536, 2048, 2056, 4095, 4096, 4104, 8192, 8200, 16384,
        16391, 20001]
TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]  # of x and of the residual stream


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(g, rows, dim, dtype, gap=0, sigma=1.0, mu=0.0):
    big = torch.full((rows, dim + gap), float("nan"), device="cuda", dtype=DT[dtype])
    big[:, :dim] = torch.randn(rows, dim, generator=g, device="cuda") * sigma + mu
    return big[:, :dim]


def f64(t):
    return t.detach().double().cpu().numpy()


def within(name, got, want, tol):
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{name}: {(~(err <= tol)).sum()} off, worst {np.nanmax(err / np.maximum(tol, 1e-300))} of the tolerance"


def check_forward(x, w, r, eps, y=None, h=None, rstd=None, codes=None, scales=None):
    want, wh, wr = orn.rms_norm_forward(f64(x), None if w is None else f64(w), None if r is None else f64(r), eps)
    d = 64 + x.shape[1] // 1024
    if h is not None:
        within("h", f64(h), wh, (U + HALF[h.dtype]) * np.abs(wh))
    if rstd is not None:
        within("rstd", f64(rstd), wr, (d + 8) * U * wr)
    tol = (d + 12) * U * np.abs(want) + 1e-40
    if y is not None:
        within("y", f64(y), want, tol + HALF[y.dtype] * (np.abs(want) + tol))
    if codes is not None:
        dim = x.shape[1]
        s = np.repeat(f64(scales), 128, 1)[:, :dim]
        got = oa.unpack(codes.cpu().numpy(), f64(scales))
        within("codes", got, want, np.maximum(2.0 ** -4 * (np.abs(want) + tol), 2.0 ** -10 * s) + tol)
        for b in range(scales.shape[1]):
            at = slice(128 * b, 128 * b + 128)
            low = [oa.scale_of(t) for t in np.maximum(np.abs(want[:, at]) - tol[:, at], 0).max(1)]
            high = [oa.scale_of(t) for t in (np.abs(want[:, at]) + tol[:, at]).max(1)]
            got_s = f64(scales)[:, b]
            assert np.all((got_s == low) | (got_s == high) | (np.abs(want[:, at]).max(1) < 1e-35))


def room(rows, dim, gap=0):
    codes = torch.full((rows, dim + gap), 0x55, device="cuda", dtype=torch.uint8)
    scales = torch.full((rows, -(-dim // 128) + gap), float("nan"), device="cuda")
    return codes, scales, codes[:, :dim], scales[:, :-(-dim // 128)]


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,stream", TYPES)
def test_forward(dim, dtype, stream):
    g = gen(dim)
    for rows, gap, wtype, with_r, out8, mu in ((1, 0, dtype, True, True, 0.0), (5, 3, "f32", True, False, 20.0),
                                               (37, 1, None, False, True, 0.5), (3, 0, "bf16", False, False, -1.0)):
        x = matrix(g, rows, dim, dtype, gap, mu=mu)
        r = matrix(g, rows, dim, stream, gap, 3.0) if with_r else None
        w = None if wtype is None else matrix(g, 1, dim, wtype, sigma=0.3, mu=1.0)[0].clone()
        y, rstd = matrix(g, rows, dim, dtype, gap), torch.full((rows,), float("nan"), device="cuda")
        h = matrix(g, rows, dim, stream, gap) if with_r else None
        big_c, big_s, codes, scales = room(rows, dim, gap) if out8 else (None,) * 4
        zs.zs_rms_norm_forward(x, w, y, eps=1e-5, residual=r, residual_out=h, codes=codes, scales=scales, rstd=rstd)
        check_forward(x, w, r, 1e-5, y, h, rstd, codes, scales)
        if out8:
            assert (big_c[:, dim:] == 0x55).all() and torch.isnan(big_s[:, scales.shape[1]:]).all()
            again = torch.empty_like(codes.contiguous())
            s2 = torch.empty_like(scales.contiguous())
            zs.zs_rms_norm_forward(x, w, None, eps=1e-5, residual=r, codes=again, scales=s2)  # in 8 bits alone
            assert torch.equal(again, codes) and torch.equal(s2, scales)


@pytest.mark.parametrize("dim", [5, 128, 1000, 4096, 8192, 20001, 40004])
@pytest.mark.parametrize("dtype,stream", TYPES)
def test_sum_in_place(dim, dtype, stream):
    g = gen(dim + 1)
    x, r = matrix(g, 9, dim, dtype, 1), matrix(g, 9, dim, stream, 2)
    w = matrix(g, 1, dim, dtype)[0].clone()
    h, y = torch.empty(9, dim, device="cuda", dtype=DT[stream]), torch.empty(9, dim, device="cuda", dtype=DT[dtype])
    zs.zs_rms_norm_forward(x, w, y, residual=r, residual_out=h)
    y2 = torch.empty_like(y)
    r2 = matrix(g, 9, dim, stream, 2)
    r2.copy_(r)
    zs.zs_rms_norm_forward(x, w, y2, residual=r2, residual_out=r2)
    assert torch.equal(r2, h) and torch.equal(y2, y)
    if dtype == stream:
        x2 = matrix(g, 9, dim, dtype, 1)
        x2.copy_(x)
        zs.zs_rms_norm_forward(x2, w, y2, residual=r, residual_out=x2)
        assert torch.equal(x2, h) and torch.equal(y2, y)


def test_rows_do_not_depend_on_their_batch():
    for dim in (96, 768, 4096, 8192):
        g = gen(dim)
        x, r = matrix(g, 700, dim, "bf16"), matrix(g, 700, dim, "bf16")
        w = matrix(g, 1, dim, "bf16")[0].clone()
        y, one = torch.empty_like(x), torch.empty(1, dim, device="cuda", dtype=torch.bfloat16)
        zs.zs_rms_norm_forward(x, w, y, residual=r)
        for i in (0, 333, 699):
            zs.zs_rms_norm_forward(x[i:i + 1], w, one, residual=r[i:i + 1])
            assert torch.equal(one[0], y[i])


def test_extreme_values():
    """Zeros, rows with one NaN or infinity (which stay in their row), tiny rows without eps."""
    dim = 300
    x = torch.ones(6, dim, device="cuda")
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 299] = float("inf")
    x[3] = 1e-15
    x[4] = 1e18
    y, rstd = torch.empty_like(x), torch.empty(6, device="cuda")
    _, _, codes, scales = room(6, dim)
    zs.zs_rms_norm_forward(x, None, y, eps=0.0 + 1e-38, codes=codes, scales=scales, rstd=rstd)
    assert (y[0] == 0).all() and (scales[0] == 1).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 299]) and (y[2, :299] == 0).all()
    for i in (3, 4, 5):
        assert torch.allclose(y[i], torch.ones(dim, device="cuda"), rtol=1e-5)
    values = oa.unpack(codes.cpu().numpy(), f64(scales))
    assert np.isnan(values[1]).all() and np.isnan(values[2, 299]) and (values[2, :299] == 0).all()
    assert np.all(np.abs(values[3:] - 1) < 0.07)


def check_backward(dy, h64, w, rstd, dres, dh, dw, old, first):
    want, wdw = orn.rms_norm_backward(f64(dy), h64, None if w is None else f64(w), f64(rstd),
                                      None if dres is None else f64(dres))
    d = 64 + dy.shape[1] // 1024
    rs = f64(rstd)[:, None]
    xh = np.abs(h64) * rs
    gw = np.abs(f64(dy)) * (1.0 if w is None else np.abs(f64(w)))
    size = rs * (gw + xh * (gw * xh).mean(1, keepdims=True))
    tol = (d + 8) * U * size + 2 * U * (size + (0.0 if dres is None else np.abs(f64(dres))))
    within("dh", f64(dh), want, tol + HALF[dh.dtype] * (np.abs(want) + tol))
    if dw is not None:
        before = np.zeros(dy.shape[1]) if first else f64(old)
        tol = (len(xh) + 6) * U * (np.abs(before) + (np.abs(f64(dy)) * xh).sum(0))
        within("dw", f64(dw), wdw + before, tol + HALF[dw.dtype] * (np.abs(wdw + before) + tol))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,stream", TYPES)
@pytest.mark.parametrize("kept8", [False, True])
def test_backward(dim, dtype, stream, kept8):
    g = gen(dim + 2)
    for rows, gap, wtype, with_r, grad, first in ((1, 0, dtype, True, "f32", True), (5, 3, "f32", True, "bf16", False),
                                                  (301, 1, None, False, "f32", False), (3, 0, "bf16", False, None, True)):
        h = matrix(g, rows, dim, stream, gap, 3.0)
        h64, scales = f64(h), None
        if kept8:
            _, _, codes, scales = room(rows, dim, gap)
            zs.zs_activation_pack(h, codes, scales)
            h, h64 = codes, oa.unpack(codes.cpu().numpy(), f64(scales))
        rstd = torch.from_numpy((1 / np.sqrt((h64 * h64).mean(1) + 1e-5)).astype(np.float32)).cuda()
        dy = matrix(g, rows, dim, dtype, gap)
        dres = matrix(g, rows, dim, stream, gap) if with_r else None
        w = None if wtype is None else matrix(g, 1, dim, wtype, sigma=0.3, mu=1.0)[0].clone()
        dh = matrix(g, rows, dim, stream, gap)
        dw = None if grad is None else matrix(g, 1, dim, grad)[0].clone()
        old = None if grad is None else dw.clone()
        size = zs.zs_rms_norm_workspace_bytes(rows, dim)
        ws = torch.full((size + 512,), 0xFF, device="cuda", dtype=torch.uint8)
        zs.zs_rms_norm_backward(dy, h, w, rstd, dh, scales=scales, dresidual=dres, dweight=dw, first=first,
                                workspace=None if grad is None else ws[:size])
        check_backward(dy, h64, w, rstd, dres, dh, dw, old, first)
        assert (ws[size:] == 0xFF).all()
        if with_r:  # in place, the same bits
            zs.zs_rms_norm_backward(dy, h, w, rstd, dres, scales=scales, dresidual=dres)
            assert torch.equal(dres, dh)


@pytest.mark.parametrize("rows,dim", [(4097, 4096), (3000, 8192), (20000, 770), (9000, 128), (1500, 20001)])
def test_many_rows(rows, dim):
    """More rows than workgroups, over the size at which accesses bypass the caches among them; the gradient twice."""
    g = gen(rows)
    h, dy, dres = (matrix(g, rows, dim, "bf16") for _ in range(3))
    w = matrix(g, 1, dim, "bf16", sigma=0.3, mu=1.0)[0].clone()
    rstd = torch.empty(rows, device="cuda")
    y = torch.empty_like(h)
    zs.zs_rms_norm_forward(h, w, y, rstd=rstd)
    ws = torch.empty(zs.zs_rms_norm_workspace_bytes(rows, dim), device="cuda", dtype=torch.uint8)
    runs = []
    for _ in range(2):
        dh, dw = torch.empty_like(h), torch.zeros(dim, device="cuda")
        zs.zs_rms_norm_backward(dy, h, w, rstd, dh, dresidual=dres, dweight=dw, first=False, workspace=ws)
        runs.append((dh, dw))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    at = torch.randint(0, rows, (16,), generator=g, device="cuda")
    check_forward(h[at], w, None, 1e-5, y[at], None, rstd[at])
    check_backward(dy[at], f64(h[at]), w, rstd[at], dres[at], dh[at], None, None, True)
    xh = h.double() * rstd.double()[:, None]
    want, size = (dy.double() * xh).sum(0), (dy.double() * xh).abs().sum(0)
    assert ((dw.double() - want).abs() <= (rows + 6) * U * size + 2.0 ** -24 * want.abs()).all()


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    zs.zs_rms_norm_forward(e, None, e.clone())
    dw = torch.ones(64, device="cuda")
    none = torch.empty(0, device="cuda")
    zs.zs_rms_norm_backward(e, e.clone(), None, none, e.clone(), dweight=dw)
    assert (dw == 1).all()
    zs.zs_rms_norm_backward(e, e.clone(), None, none, e.clone(), dweight=dw, first=True)
    assert (dw == 0).all()
