"""Layer norm's forward and backward pass against the fp64 oracle.

Tolerances, u = 2^-24, h = half a step of the result's type (2^-24 fp32,
2^-8 bf16), d = the most additions on the way of one element in a sum over a
row. A lane adds up to 32 elements of a row (dim / 1024 for rows that do not
fit in registers), then come at most 6 + 16 + 2 joins over lanes and waves:
d = 64 + dim / 1024 covers it. With A = mean |x|, xh = (x - mean) rstd:
  mean:  |err| <= (d + 2) u A
  rstd:  the squares' sum is relative to itself, (d + 4) u, and the mean's error
         e = (d + 2) u A enters with e^2 rstd^2 (the linear term cancels up to
         another rounding) and through each rounded difference: relative
         (d + 8) u + (e rstd)^2 + 2 u e rstd
  y:     |w| (e rstd + |xh| (r + 3 u)) + 2 u (|xh w| + |b|) + h |y|, r the bound above
  dx:    with g = dy w, S = rstd (|g| + mean |g| + |xh| mean |g xh|), statistics as
         given: every term carries at most d + 8 roundings: (d + 8) u S + h |dx|
  dw:    (rows + 6) u (|old| + sum |dy xh|) + h |dw|;  db alike
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
DIMS = [1, 2, 7, 64, 127, 128, 129, 257, 512, 513, 768, 1024, 1031, 2048, 2056, 4095, 4096, 4104, 8192, 8200, 10240,
        16384, 16391, 20001, 33003]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def matrix(g, rows, dim, dtype, gap=0, mu=0.0, fill=None):
    big = torch.full((rows, dim + gap), float("nan"), device="cuda", dtype=DT[dtype])
    v = big[:, :dim]
    v.copy_(torch.randn(rows, dim, generator=g, device="cuda") + mu if fill is None else torch.full((), fill))
    return big, v


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)


def within(name, got, want, tol):
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"{name}: {(err > tol).sum()} off, worst {np.max(err / np.maximum(tol, 1e-300))} of the tolerance"


def check_forward(x, w, b, y, mean, rstd, eps):
    xd = f64(x)
    wd, bd = (None if t is None else f64(t) for t in (w, b))
    want, m, r = ol.layer_norm_forward(xd, wd, bd, eps)
    d = 64 + x.shape[1] // 1024
    e = (d + 2) * U * np.abs(xd).mean(1)
    rel = (d + 8) * U + (e * r) ** 2 + 2 * U * e * r
    if mean is not None:
        within("mean", mean, m, e)
    if rstd is not None:
        within("rstd", rstd, r, rel * r)
    xh = np.abs(xd - m[:, None]) * r[:, None]
    wa, ba = (1.0 if wd is None else np.abs(wd)), (0.0 if bd is None else np.abs(bd))
    tol = wa * ((e * r)[:, None] + xh * (rel + 3 * U)[:, None]) + 2 * U * (xh * wa + ba)
    within("y", y, want, (tol + HALF[y.dtype] * np.abs(want)) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_forward(dim, dtype, wdtype):
    g = gen(dim)
    for rows, gap, affine, mu in ((1, 0, "wb", 0.0), (5, 3, "w", 20.0), (37, 1, "", 0.5), (3, 0, "b", -1.0)):
        _, x = matrix(g, rows, dim, dtype, gap, mu)
        big, y = matrix(g, rows, dim, dtype, 2 * gap, fill=float("nan"))
        w = matrix(g, 1, dim, wdtype)[1][0] if "w" in affine else None
        b = matrix(g, 1, dim, wdtype)[1][0] if "b" in affine else None
        mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
        zs.zs_layer_norm_forward(x, w, b, y, eps=1e-5, mean=mean, rstd=rstd)
        check_forward(x, w, b, y, mean, rstd, 1e-5)
        assert torch.isnan(big[:, dim:]).all()
        again = torch.empty(rows, dim, device="cuda", dtype=DT[dtype])
        zs.zs_layer_norm_forward(x, w, b, again, eps=1e-5)  # without the statistics, to another stride
        assert torch.equal(bits(again), bits(y))


@pytest.mark.parametrize("dim,rows", [(64, 70001), (768, 9000), (4096, 5001), (8192, 2500), (16400, 2100)])
def test_forward_many_rows(dim, rows):
    # more rows than workgroups: every row equals the same row computed alone
    g = gen(rows)
    _, x = matrix(g, rows, dim, "bf16")
    w, b = matrix(g, 1, dim, "bf16")[1][0], matrix(g, 1, dim, "bf16")[1][0]
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zs.zs_layer_norm_forward(x, w, b, y, mean=mean, rstd=rstd)
    pick = torch.tensor([0, 1, rows // 3, rows // 2 + 1, rows - 2, rows - 1], device="cuda")
    check_forward(x[pick], w, b, y[pick], mean[pick], rstd[pick], 1e-5)
    one = torch.empty(1, dim, device="cuda", dtype=torch.bfloat16)
    for i in pick.tolist():
        zs.zs_layer_norm_forward(x[i:i + 1], w, b, one)
        assert torch.equal(bits(one[0]), bits(y[i]))


def test_forward_degenerate_rows():
    dim = 700
    x = torch.zeros(6, dim, device="cuda")
    x[1] = 1.0  # constant rows: variance 0
    x[2] = 3.0e4
    x[3] = torch.randn(dim, device="cuda")
    x[3, 9] = float("inf")
    x[4] = torch.randn(dim, device="cuda")
    x[4, 11] = float("nan")
    x[5] = torch.randn(dim, device="cuda")
    w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    zs.zs_layer_norm_forward(x, w, b, y, eps=1e-5, mean=mean, rstd=rstd)
    for i in (0, 1):
        assert torch.equal(y[i], b) and mean[i] == i  # 700 ones add up exactly
        assert abs(float(rstd[i]) * 1e-5 ** 0.5 - 1) < 4 * U  # eps, its root and the quotient round
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.isfinite(y[5]).all() and torch.isfinite(y[2]).all()
    check_forward(x[5:], w, b, y[5:], mean[5:], rstd[5:], 1e-5)
    zs.zs_layer_norm_forward(x[:1], w, b, y[:1], eps=0.0, rstd=rstd[:1])
    assert torch.isinf(rstd[0]) and torch.isnan(y[0]).all()  # 0 * (1 / 0)


def test_no_rows():
    x = torch.empty(0, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    z = torch.empty(0, device="cuda")
    zs.zs_layer_norm_forward(x, w, w, x.clone(), mean=z, rstd=z.clone())
    dw, db = torch.full((16,), 3.0, device="cuda"), torch.full((16,), float("nan"), device="cuda")
    zs.zs_layer_norm_backward(x, x.clone(), w, z, z.clone(), x.clone(), dweight=dw, dbias=db)
    assert torch.all(dw == 3.0)
    zs.zs_layer_norm_backward(x, x.clone(), w, z, z.clone(), x.clone(), dweight=dw, dbias=db, first=True)
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def stats(x, eps=1e-5):
    m = x.float().mean(1)
    return m, ((x.float() - m[:, None]) ** 2).mean(1).add(eps).rsqrt()


def run_backward(dy, x, w, mean, rstd, dx, dw, db, first):
    ws = torch.full((zs.zs_layer_norm_workspace_bytes(*x.shape),), 0xFF, device="cuda", dtype=torch.uint8)  # NaN
    zs.zs_layer_norm_backward(dy, x, w, mean, rstd, dx, dweight=dw, dbias=db, first=first, workspace=ws)


def check_backward(dy, x, w, mean, rstd, dx, dw, db, old_w, old_b):
    rows, dim = x.shape
    wd = None if w is None else f64(w)
    want = ol.layer_norm_backward(f64(dy), f64(x), wd, f64(mean), f64(rstd))
    r = f64(rstd)[:, None]
    xh = np.abs(f64(x) - f64(mean)[:, None]) * r
    dya = np.abs(f64(dy))
    ga = dya if wd is None else dya * np.abs(wd)
    s = r * (ga + ga.mean(1, keepdims=True) + xh * (ga * xh).mean(1, keepdims=True))
    d = 64 + dim // 1024
    within("dx", dx, want[0], ((d + 8) * U * s + HALF[dx.dtype] * np.abs(want[0])) * (1 + 2.0 ** -7))
    for name, got, total, size, old in (("dweight", dw, want[1], (dya * xh).sum(0), old_w),
                                        ("dbias", db, want[2], dya.sum(0), old_b)):
        if got is None:
            continue
        if old is not None:
            total, size = total + f64(old), size + np.abs(f64(old))
        within(name, got, total, ((rows + 6) * U * size + HALF[got.dtype] * np.abs(total)) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_backward(dim, dtype, wdtype):
    g = gen(dim + 1)
    for k, (rows, gap) in enumerate(((1, 0), (6, 3), (41, 1))):
        _, x = matrix(g, rows, dim, dtype, gap, 0.5)
        _, dy = matrix(g, rows, dim, dtype, 2 * gap)
        big, dx = matrix(g, rows, dim, dtype, gap, fill=float("nan"))
        w = matrix(g, 1, dim, wdtype)[1][0] if k else None
        mean, rstd = stats(x)
        gdt = ("f32", "bf16", "f32")[k]
        first = k != 2
        dw, db = (matrix(g, 1, dim, gdt, fill=float("nan") if first else None)[1][0] for _ in range(2))
        old = (None, None) if first else (dw.clone(), db.clone())
        run_backward(dy, x, w, mean, rstd, dx, dw, db, first)
        check_backward(dy, x, w, mean, rstd, dx, dw, db, *old)
        assert torch.isnan(big[:, dim:]).all()
        # one gradient alone, then none: the same dx
        dw2, dx2 = torch.empty_like(dw), torch.empty(rows, dim, device="cuda", dtype=DT[dtype])
        if first:
            run_backward(dy, x, w, mean, rstd, dx2, dw2, None, True)
            assert torch.equal(bits(dw2), bits(dw)) and torch.equal(bits(dx2), bits(dx))
            run_backward(dy, x, w, mean, rstd, dx2, None, dw2, True)
            assert torch.equal(bits(dw2), bits(db))
        zs.zs_layer_norm_backward(dy, x, w, mean, rstd, dx2)
        assert torch.equal(bits(dx2), bits(dx))


@pytest.mark.parametrize("dim,rows", [(64, 30000), (130, 5000), (768, 3000), (1601, 1201), (4096, 1500), (8192, 700),
                                      (16390, 600)])
def test_backward_many_rows(dim, rows):
    g = gen(rows + 1)
    for dtype in ("bf16", "f32"):
        _, x = matrix(g, rows, dim, dtype)
        _, dy = matrix(g, rows, dim, dtype)
        w = matrix(g, 1, dim, dtype)[1][0]
        mean, rstd = stats(x)
        dx = torch.empty_like(x)
        dw, db = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
        old = dw.clone(), db.clone()
        run_backward(dy, x, w, mean, rstd, dx, dw, db, False)
        check_backward(dy, x, w, mean, rstd, dx, dw, db, *old)
        dw2, db2 = (t.clone() for t in old)
        run_backward(dy, x, w, mean, rstd, dx, dw2, db2, False)  # the same bits again
        assert torch.equal(bits(dw2), bits(dw)) and torch.equal(bits(db2), bits(db))


@pytest.mark.parametrize("rows,dim,dtype", [(4099, 8192, "bf16"), (9001, 1601, "f32")])
def test_large_calls_past_the_caches(rows, dim, dtype):
    # more than 100 MB: the streaming variants, against the same rows in smaller calls
    g = gen(dim)
    _, x = matrix(g, rows, dim, dtype, 0, 0.25)
    _, dy = matrix(g, rows, dim, dtype)
    w, b = matrix(g, 1, dim, dtype)[1][0], matrix(g, 1, dim, dtype)[1][0]
    y, dx, y2, dx2 = (torch.empty_like(x) for _ in range(4))
    mean, rstd, mean2, rstd2 = (torch.empty(rows, device="cuda") for _ in range(4))
    dw, db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    zs.zs_layer_norm_forward(x, w, b, y, mean=mean, rstd=rstd)
    run_backward(dy, x, w, mean, rstd, dx, dw, db, True)
    for i in range(0, rows, 1000):
        j = slice(i, i + 1000)
        zs.zs_layer_norm_forward(x[j], w, b, y2[j], mean=mean2[j], rstd=rstd2[j])
        zs.zs_layer_norm_backward(dy[j], x[j], w, mean[j], rstd[j], dx2[j])
    for p, q in ((y, y2), (mean, mean2), (rstd, rstd2), (dx, dx2)):
        assert torch.equal(bits(p), bits(q))
    check_forward(x[:50], w, b, y[:50], mean[:50], rstd[:50], 1e-5)
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    for got, terms in ((dw, dy.double() * xh), (db, dy.double())):
        err = (got.double() - terms.sum(0)).abs()
        assert bool((err <= (rows + 6) * U * terms.abs().sum(0) * (1 + 2.0 ** -7)).all())


def test_backward_against_differences():
    # fp32 at small sizes: the loss sum(y c) along a direction v, from the library's own forward pass
    g = gen(3)
    rows, dim = 3, 24
    x, c, v = (torch.randn(rows, dim, generator=g, device="cuda") for _ in range(3))
    w, b = torch.randn(dim, generator=g, device="cuda"), torch.randn(dim, generator=g, device="cuda")
    y, mean, rstd, dx = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    zs.zs_layer_norm_forward(x, w, b, y, mean=mean, rstd=rstd)
    run_backward(c, x, w, mean, rstd, dx, dw, db, True)

    def loss(x, w, b):
        zs.zs_layer_norm_forward(x, w, b, y)
        return float((y.double() * c.double()).sum())

    # central differences: the third derivative's term h^2 / 6 and the outputs' rounding, 72 terms of
    # a few u each over h, are both below 1e-3 of values of order 1 at h = 2^-7
    h = 2.0 ** -7
    for grad, args in ((dx, lambda t: (x + t * v, w, b)), (dw, lambda t: (x, w + t * v[0], b)), (db, lambda t: (x, w, b + t * v[0]))):
        direction = v if grad is dx else v[0]
        want = float((grad.double() * direction.double()).sum())
        got = (loss(*args(h)) - loss(*args(-h))) / (2 * h)
        scale = float((grad.abs().double() * direction.abs().double()).sum())
        assert abs(got - want) <= 2e-2 * scale if grad is dx else abs(got - want) <= 1e-3 * scale


def test_backward_non_finite_rows():
    g = gen(4)
    _, x = matrix(g, 9, 300, "f32")
    _, dy = matrix(g, 9, 300, "f32")
    mean, rstd = stats(x)
    w = torch.ones(300, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    dy[4, 7] = float("nan")
    run_backward(dy, x, w, mean, rstd, dx, dw, db, True)
    rows = torch.isnan(dx).all(1)
    assert rows.tolist() == [False] * 4 + [True] + [False] * 4 and torch.isfinite(dx[~rows]).all()
    for t in (dw, db):
        assert torch.isnan(t[7]) and torch.isfinite(t).sum() == 299


def test_rows_beyond_32_bits():
    ld, rows, dim = 1 << 22, 600, 200
    x = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16).view(rows, ld)[:, :dim]
    x.copy_(torch.randn(rows, dim, device="cuda"))
    near = x.contiguous()
    w, b = torch.randn(dim, device="cuda"), torch.randn(dim, device="cuda")
    y, yn = torch.empty_like(near), torch.empty_like(near)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zs.zs_layer_norm_forward(x, w, b, y, mean=mean, rstd=rstd)
    zs.zs_layer_norm_forward(near, w, b, yn)
    assert torch.equal(bits(y), bits(yn))
    dw, db, dw2, db2 = (torch.empty(dim, device="cuda") for _ in range(4))
    dxn = torch.empty_like(near)
    run_backward(y, near, w, mean, rstd, dxn, dw, db, True)
    dx = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16).view(rows, ld)[:, :dim]
    run_backward(y, x, w, mean, rstd, dx, dw2, db2, True)
    assert torch.equal(bits(dx), bits(dxn)) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_widest_rows_and_many_rows():
    g = gen(9)
    dim = 2 ** 24 - 1
    _, x = matrix(g, 2, dim, "f32", 0, 1.0)
    _, dy = matrix(g, 2, dim, "f32")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    dw, db = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    zs.zs_layer_norm_forward(x, None, None, y, mean=mean, rstd=rstd)
    check_forward(x, None, None, y, mean, rstd, 1e-5)
    run_backward(dy, x, None, mean, rstd, dx, dw, db, True)
    check_backward(dy, x, None, mean, rstd, dx, dw, db, None, None)
    # 40 million rows of two: y is +-1 up to eps, and the gradients' sums of whole numbers are exact
    rows = 40_000_003
    x = torch.tensor([[-1.0, 1.0]], device="cuda").repeat(rows, 1)
    y = torch.empty_like(x)
    zs.zs_layer_norm_forward(x, None, None, y, eps=0.0)
    assert torch.equal(y, x)
    dy = torch.randint(-1, 2, (rows, 2), generator=g, device="cuda").float()
    ones, zeros = torch.ones(rows, device="cuda"), torch.zeros(rows, device="cuda")
    dw, db = torch.empty(2, device="cuda"), torch.empty(2, device="cuda")
    run_backward(dy, x, None, zeros, ones, y, dw, db, True)
    assert torch.equal(db.double(), dy.double().sum(0)) and torch.equal(dw.double(), (dy * x).double().sum(0))


def test_streams_and_graph_replays():
    g = gen(6)
    rows, dim = 900, 1032
    _, x = matrix(g, rows, dim, "bf16")
    _, dy = matrix(g, rows, dim, "bf16")
    w, b = matrix(g, 1, dim, "bf16")[1][0], matrix(g, 1, dim, "bf16")[1][0]

    def bufs():
        return dict(y=torch.empty_like(x), mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"),
                    dx=torch.empty_like(x), dw=torch.zeros(dim, device="cuda"), db=torch.zeros(dim, device="cuda"),
                    ws=torch.empty(zs.zs_layer_norm_workspace_bytes(rows, dim), device="cuda", dtype=torch.uint8))

    def both(o, stream=None):
        zs.zs_layer_norm_forward(x, w, b, o["y"], mean=o["mean"], rstd=o["rstd"], stream=stream)
        zs.zs_layer_norm_backward(dy, x, w, o["mean"], o["rstd"], o["dx"], dweight=o["dw"], dbias=o["db"],
                                  workspace=o["ws"], stream=stream)

    def same(p, q):
        return all(torch.equal(bits(p[k]), bits(q[k])) for k in ("y", "mean", "rstd", "dx", "dw", "db"))

    a, e, c = bufs(), bufs(), bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(a)
    for it in range(4):
        x.copy_(torch.randn(rows, dim, generator=g, device="cuda"))
        both(e)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(a, e), it
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for t in ("dw", "db"):
        c[t].zero_()
        e[t].zero_()
    torch.cuda.synchronize()
    both(c, s1)
    both(e, s2)
    torch.cuda.synchronize()
    assert same(c, e)


def test_refusals_of_the_binding():
    x, y = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda")
    w, m = torch.zeros(8, device="cuda"), torch.zeros(4, device="cuda")
    r, dx = m.clone(), torch.zeros(4, 8, device="cuda")
    ws = torch.empty(1 << 16, device="cuda", dtype=torch.uint8)
    for args, kw in [((x, w, w, x), {}), ((x, w[:7], w, y), {}), ((x, w, w.bfloat16(), y), {}), ((x, w, w, y[:3]), {}),
                     ((x, w, w, y.bfloat16()), {}), ((x.half(), w, w, y.half()), {}), ((x, w.half(), None, y), {}),
                     ((x, w.cpu(), w, y), {}), ((x, w, w, y), dict(mean=m[:3])), ((x, w, w, y), dict(rstd=m.double())),
                     ((x, w, w, y), dict(eps=-1.0)), ((x, w, w, y), dict(mean=m, rstd=m)), ((x.t(), w[:4], None, y.t()), {})]:
        with pytest.raises(ValueError):
            zs.zs_layer_norm_forward(*args, **kw)
    dw, db = torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    for args, kw in [((y, x, w, m, r, x), {}), ((y, x, w, m, r, y), {}), ((y, x, w, None, r, dx), {}),
                     ((y[:3], x, w, m, r, dx), {}), ((y, x, w, m, r, dx), dict(dweight=dw)),
                     ((y, x, w, m, r, dx), dict(dweight=dw, workspace=ws[:16])),
                     ((y, x, w, m, r, dx), dict(dweight=dw, dbias=db.bfloat16(), workspace=ws)),
                     ((y, x, w, m, r, dx), dict(dweight=dw, dbias=dw, workspace=ws)),
                     ((y, x, w, m, r, dx), dict(dweight=w, workspace=ws)), ((y, x, w[:4], m, r, dx), {})]:
        with pytest.raises(ValueError):
            zs.zs_layer_norm_backward(*args, **kw)
