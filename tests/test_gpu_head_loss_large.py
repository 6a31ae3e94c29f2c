"""The loss over a vocabulary at sizes of many tiles, several pieces and offsets
past 32 bits, its edges without tokens, and calls on streams and in graphs.

Large sizes are checked on samples, with the bounds of test_gpu_head_loss: some
tokens against the whole vocabulary, some rows of the head against all tokens.
"""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_flatparameter_amd as zs
from oracle import head_loss as oh
from test_gpu_head_loss import DT, HALF, U, bits, bounds, check_backward, check_forward, e_of, f64, gen, labels_of, matrix, scratch, sums, within

pytestmark = pytest.mark.gpu


def forward(h, w, t, dtype):
    n = len(h)
    big, ws = scratch(n, len(w), h.shape[1], dtype)
    loss, lse = (torch.full((n,), float("nan"), device="cuda") for _ in range(2))
    zs.zs_linear_cross_entropy_forward(h, w, t, loss, lse=lse, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all()
    return loss, lse


def check_sampled(h, w, t, lse, scale, dh, dw, old, first, tokens, rows):
    f32, grad32 = h.dtype == torch.float32, dw.dtype == torch.float32
    n, vocab = len(h), len(w)
    segments = 6 if f32 else 1
    extra = 2.0 ** -21 if f32 else 0.0
    labels = t.cpu().numpy().astype(np.int64)
    # dh of some tokens
    hs, wd, ts, ls = f64(h[tokens]), f64(w), labels[tokens], f64(lse[tokens])
    live = oh.counted(ts, vocab)
    want, _, g = oh.loss_backward(hs, wd, ts, ls, np.full(len(ts), scale))
    z, e = bounds(hs[live], wd, f32)
    x = z - ls[live][:, None]
    p = np.exp(x)
    dg = abs(scale) * (p * (1.01 * e + e_of(x)) + 3 * U * (p + 1))
    ag = np.abs(g[live])
    r = 2.0 ** -23 if f32 else 2.0 ** -8
    tol = (dg + r * ag) @ np.abs(wd) + (sums(vocab, segments) + 64 * U + extra) * (ag @ np.abs(wd))
    got = f64(dh[tokens])
    within("dh", got[live], want[live], tol + HALF[dh.dtype] * (np.abs(want[live]) + tol))
    assert np.all(got[~live] == 0)
    # dw of some rows
    live = oh.counted(labels, vocab)
    hd, lsd, lab = f64(h)[live], f64(lse)[live], labels[live]
    ws = f64(w[rows])
    z, e = bounds(hd, ws, f32)
    x = z - lsd[:, None]
    p = np.exp(x)
    g = scale * (p - (lab[:, None] == rows[None, :]))
    dg = abs(scale) * (p * (1.01 * e + e_of(x)) + 3 * U * (p + 1))
    r = 2.0 ** -23 if f32 else 2.0 ** -16 if grad32 else 2.0 ** -8
    extra = extra if grad32 else 2.0 ** -13 if f32 else 0.0
    before = np.zeros((len(rows), h.shape[1])) if first else f64(old[rows])
    want = g.T @ hd + before
    tol = (dg + r * np.abs(g)).T @ np.abs(hd) + (sums(n, 6 if f32 else 2) + 64 * U + extra) * (np.abs(g).T @ np.abs(hd))
    tol += 2 * U * np.abs(before)
    within("dw", f64(dw[rows]), want, tol + HALF[dw.dtype] * (np.abs(want) + tol))


# the widest tiles with ragged edges; pieces of the vocabulary (33000 tokens: three); splits; few and many tokens
@pytest.mark.parametrize("n,vocab,dim,dtype,grad,first,ignored", [
    (1100, 33000, 192, "bf16", "bf16", True, 0.0),
    (1029, 20001, 264, "bf16", "f32", False, 0.3),
    (700, 18000, 130, "f32", "f32", True, 0.3),
    (33000, 20011, 64, "bf16", "f32", True, 0.1),
    (40, 50257, 768, "bf16", "f32", False, 0.0),
    (17, 30011, 512, "f32", "bf16", True, 0.0),
    (5, 128256, 1024, "bf16", "bf16", True, 0.0),
    (3, 40009, 777, "f32", "f32", False, 0.0),
    (20000, 9001, 96, "f32", "f32", False, 0.2),
    (100, 50021, 1000, "f32", "bf16", True, 0.0),
    (64, 30001, 1027, "f32", "f32", False, 0.4),
])
def test_large(n, vocab, dim, dtype, grad, first, ignored):
    g = gen(n + vocab)
    w = matrix(g, vocab, dim, dtype, 0, 0.1)[1]
    h = matrix(g, n, dim, dtype)[1]
    t = labels_of(g, n, vocab, torch.int64, ignored)
    live = (t >= 0) & (t < vocab)
    h[~live] = float("nan")
    loss, lse = forward(h, w, t, dtype)
    rng = np.random.default_rng(n)
    tokens = np.unique(np.concatenate([rng.integers(0, n, 12), [0, n - 1]]))
    check_forward(h[tokens], w, t[tokens], loss[tokens], lse[tokens])
    dh = matrix(g, n, dim, dtype)[1]
    dw = matrix(g, vocab, dim, grad, 0, 1e-3)[1]
    old = dw.clone()
    big, ws = scratch(n, vocab, dim, dtype, grad)
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, scale=1.0 / n, first=first, workspace=ws)
    assert (big[ws.numel():] == 0xFF).all()
    some = t[live][:6].cpu().numpy()
    rows = np.unique(np.concatenate([rng.integers(0, vocab, 12), [0, vocab - 1], some]))
    check_sampled(h, w, t, lse, np.float64(np.float32(1.0 / n)), dh, dw, old, first, tokens, rows)
    # the same call gives the same bits, whatever the workspace held
    ws.fill_(0x5A)
    dh2, dw2 = torch.empty_like(dh), old.clone()
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh2, dw2, scale=1.0 / n, first=first, workspace=ws)
    assert torch.equal(bits(dh2), bits(dh)) and torch.equal(bits(dw2), bits(dw))
    loss2, lse2 = forward(h, w, t, dtype)
    assert torch.equal(bits(loss2), bits(loss)) and torch.equal(bits(lse2), bits(lse))


@pytest.mark.parametrize("n", [2, 40, 300])
def test_offsets_past_32_bits(n):
    """A head of 4.9 GB, read to its last row; its gradient's last rows."""
    vocab, dim = 300007, 8192
    g = gen(n)
    w = torch.empty(vocab, dim, device="cuda", dtype=torch.bfloat16).normal_(0, 0.05, generator=g)
    h = matrix(g, n, dim, "bf16")[1]
    t = torch.randint(vocab - 1000, vocab, (n,), generator=g, device="cuda")
    t[0] = vocab - 1
    loss, lse = forward(h, w, t, "bf16")
    z = torch.cat([h[:2].double() @ w[v:v + 20000].double().t() for v in range(0, vocab, 20000)], 1)
    want = torch.logsumexp(z, 1)
    # logits of |h w| = 0.05 * 8192 * 0.8^2 in sums(8192): 2 (32 + 256) 2^-24 * 262
    assert ((lse[:2].double() - want).abs() < 0.02).all()
    assert ((loss[:2].double() - (want - z.gather(1, t[:2, None])[:, 0])).abs() < 0.04).all()
    dw = torch.empty_like(w)
    dh = torch.empty_like(h)
    ws = torch.empty(zs.zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, torch.bfloat16, torch.bfloat16), device="cuda",
                     dtype=torch.uint8)
    zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, first=True, workspace=ws)
    rows = np.array([0, 1, 262144, vocab - 2, vocab - 1])
    check_sampled(h, w, t, lse, 1.0, dh, dw, dw, True, np.array([], np.int64), rows)


def test_wide_stride():
    """Rows further apart than 32 bits of offset reach for a tile are laid out first."""
    ld, vocab, dim = (1 << 22) + 64, 70, 64
    g = gen(3)
    flat = torch.zeros(ld * vocab, device="cuda", dtype=torch.bfloat16)
    w = flat.view(vocab, ld)[:, :dim]
    w.copy_(torch.randn(vocab, dim, generator=g, device="cuda"))
    for n in (9, 70, 300):
        h = matrix(g, n, dim, "bf16")[1]
        t = labels_of(g, n, vocab, torch.int32, 0.0)
        loss, lse = forward(h, w, t, "bf16")
        check_forward(h, w, t, loss, lse)
        dh, dw = torch.empty(n, dim, device="cuda", dtype=torch.bfloat16), torch.empty(vocab, dim, device="cuda")
        _, ws = scratch(n, vocab, dim, "bf16", "f32")
        zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, first=True, workspace=ws)
        check_backward(h, w, t, lse, np.ones(n), dh, dw, dw, True)


@pytest.mark.parametrize("n", [1, 16, 20, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_token_counts(n, dtype):
    g = gen(n)
    w, h = matrix(g, 500, 64, dtype)[1], matrix(g, n, 64, dtype)[1]
    h[:] = float("nan")
    t = torch.full((n,), -100, device="cuda")
    loss, lse = forward(h, w, t, dtype)
    assert (loss == 0).all() and (lse == 0).all()
    for first in (True, False):
        dh, dw = torch.full_like(h, 7.0), torch.full((500, 64), 3.0, device="cuda")
        _, ws = scratch(n, 500, 64, dtype, "f32")
        zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, first=first, workspace=ws)
        assert (dh == 0).all() and (dw == (0.0 if first else 3.0)).all()


def test_no_tokens_and_no_vocabulary():
    w, e = torch.ones(9, 4, device="cuda"), torch.empty(0, 4, device="cuda")
    none, ids = torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=torch.int64)
    zs.zs_linear_cross_entropy_forward(e, w, ids, none, workspace=None)
    dw = torch.ones(9, 4, device="cuda")
    zs.zs_linear_cross_entropy_backward(e, w, ids, none, e.clone(), dw, workspace=None)
    assert (dw == 1).all()
    zs.zs_linear_cross_entropy_backward(e, w, ids, none, e.clone(), dw, first=True, workspace=None)
    assert (dw == 0).all()
    for n in (3, 400):
        h, t = torch.ones(n, 4, device="cuda"), torch.zeros(n, device="cuda", dtype=torch.int64)
        loss, lse = forward(h, e, t, "f32")
        assert (loss == 0).all() and (lse == 0).all()
        dh = torch.ones_like(h)
        zs.zs_linear_cross_entropy_backward(h, e, t, lse, dh, e.clone(), first=True, workspace=None)
        assert (dh == 0).all()


@pytest.mark.parametrize("n", [6, 60, 400])
def test_nonfinite_values_stay_in_their_token(n):
    g = gen(n)
    w, h = matrix(g, 700, 64, "bf16", 0, 0.3)[1], matrix(g, n, 64, "bf16")[1]
    t = labels_of(g, n, 700, torch.int64, 0.0)
    clean = forward(h, w, t, "bf16")
    h[2, 5], h[4, 0] = float("inf"), float("nan")
    loss, lse = forward(h, w, t, "bf16")
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[[2, 4]] = False
    assert torch.equal(loss[keep], clean[0][keep]) and not torch.isfinite(loss[~keep]).any()
    w[3] = float("-inf")  # a row of the head that is switched off for hidden states of one sign
    h = h.abs()
    h[2, 5] = h[4, 0] = 1.0
    t[t == 3] = 4
    loss, lse = forward(h, w, t, "bf16")
    w[3] = -1000.0
    same, _ = forward(h, w, t, "bf16")
    assert torch.isfinite(loss).all() and torch.allclose(loss, same, rtol=1e-6, atol=1e-6)


def test_against_differences():
    rng = np.random.default_rng(5)
    n, vocab, dim = 6, 11, 5
    h, w = rng.standard_normal((n, dim)).astype(np.float32), rng.standard_normal((vocab, dim)).astype(np.float32)
    t, c = np.array([0, 10, -1, 4, 4, 7]), rng.standard_normal(n).astype(np.float32)
    dev = [torch.from_numpy(a).cuda() for a in (h, w, t, c)]
    _, lse = forward(dev[0], dev[1], dev[2], "f32")
    dh, dw = torch.empty(n, dim, device="cuda"), torch.empty(vocab, dim, device="cuda")
    _, ws = scratch(n, vocab, dim, "f32", "f32")
    zs.zs_linear_cross_entropy_backward(dev[0], dev[1], dev[2], lse, dh, dw, dloss=dev[3], scale=0.5, first=True, workspace=ws)
    h, w, e = h.astype(np.float64), w.astype(np.float64), 1e-5
    for a, d in ((h, f64(dh)), (w, f64(dw))):
        for at in np.ndindex(a.shape):
            a[at] += e
            up = (oh.loss_forward(h, w, t)[0] * c * 0.5).sum()
            a[at] -= 2 * e
            down = (oh.loss_forward(h, w, t)[0] * c * 0.5).sum()
            a[at] += e
            # differences are good to e^2 and 1e-16 / e; the gradient to 100 u of terms below 10
            assert abs((up - down) / (2 * e) - d[at]) < 1e-8 + 1000 * U


@pytest.mark.parametrize("n,vocab,dim,dtype", [
    (600, 3000, 192, "bf16"), (7, 3000, 100, "bf16"), (300, 1000, 100, "f32"), (100, 700, 2048, "bf16"), (2000, 90, 130, "f32"),
    (50, 3000, 100, "f32")])
def test_graph_and_streams(n, vocab, dim, dtype):
    """Captured forward and backward passes on a stream of their own, replayed with new inputs, with other calls on
    another stream and workspace at the same time."""
    g = gen(n)
    w, h = matrix(g, vocab, dim, dtype, 0, 0.1)[1], matrix(g, n, dim, dtype)[1]
    t = labels_of(g, n, vocab, torch.int64, 0.2)
    grad = torch.float32
    ws, ws2 = (torch.empty(max(zs.zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, DT[dtype]),
                               zs.zs_linear_cross_entropy_workspace_bytes(n, vocab, dim, DT[dtype], grad)), device="cuda",
                           dtype=torch.uint8) for _ in range(2))

    def buffers():
        return (torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, dim, device="cuda", dtype=DT[dtype]),
                torch.zeros(vocab, dim, device="cuda"))

    def both(out, work, stream=None):
        loss, lse, dh, dw = out
        zs.zs_linear_cross_entropy_forward(h, w, t, loss, lse=lse, workspace=work, stream=stream)
        zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, scale=0.1, workspace=work, stream=stream)

    captured, eager = buffers(), buffers()
    both(eager, ws2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(captured, ws)
    side = torch.cuda.Stream()
    for turn in range(4):
        h.copy_(torch.randn(n, dim, generator=g, device="cuda"))
        t.copy_(labels_of(g, n, vocab, torch.int64, 0.2 * turn))  # other numbers of tokens count
        for b in (captured, eager):
            b[3].zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            both(eager, ws2)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(bits(a), bits(b))
    check_forward(h, w, t, captured[0], captured[1])


@pytest.mark.parametrize("n,vocab,dim", [(65, 301, 97), (300, 1000, 200)])
def test_fp32_rows_of_any_magnitude(n, vocab, dim):
    """Rows scaled from 2^-100 to 2^100, their columns over 12 decades, zero rows, an infinite one."""
    rng = np.random.default_rng(n)
    up = rng.integers(-100, 101, n)
    h = rng.standard_normal((n, dim)) * 10.0 ** rng.uniform(-6, 6, dim)
    h = np.ldexp(h / np.abs(h).max(1)[:, None], up[:, None])
    w = rng.standard_normal((vocab, dim)) * 10.0 ** rng.uniform(-6, 6, dim)
    w /= np.abs(w).max(1)[:, None]
    h, w = h.astype(np.float32), w.astype(np.float32)
    h[7], w[9] = 0.0, 0.0
    h[8] = np.float32(2.0 ** -140)  # subnormal throughout
    keep = up <= 3                  # of larger rows the logits' own size leaves no digits to compare
    keep[[7, 8]] = True
    t = rng.integers(0, vocab, n)
    loss, lse = forward(torch.from_numpy(h).cuda(), torch.from_numpy(w).cuda(), torch.from_numpy(t).cuda(), "f32")
    h, w = h.astype(np.float64), w.astype(np.float64)
    want_loss, want_lse = oh.loss_forward(h, w, t)
    a, b = np.abs(h), np.abs(w)
    # each product within 3 2^-22 of itself and 2^-39 of |h| max|w| and |w| max|h|; sums of 32 products round twice a product at most
    e = (3 * 2.0 ** -22 + 2 * (32 + 3 * dim / 32) * U) * (a @ b.T)
    e += 2.0 ** -39 * (a.sum(1)[:, None] * b.max(1) + a.max(1)[:, None] * b.sum(1))
    z = h @ w.T
    top = z.max(1)
    rest = 2 * ((top - z.min(1)) + 4) * 2.0 ** -23 + (128 + vocab / 1024) * U + 4 * U * (np.abs(top) + np.log(vocab))
    assert np.isfinite(f64(loss)).all()
    assert (np.abs(f64(lse) - want_lse) <= e.max(1) + rest)[keep].all()
    assert (np.abs(f64(loss) - want_loss) <= 2 * e.max(1) + rest)[keep].all()


def test_fp32_rows_of_minus_infinity():
    g = gen(3)
    w, h = matrix(g, 700, 100, "f32", 0, 0.3)[1], matrix(g, 300, 100, "f32")[1].abs()
    t = labels_of(g, 300, 700, torch.int64, 0.0)
    t[t == 3] = 4
    w[3] = float("-inf")
    w[3, 50:] = -1e38
    loss, _ = forward(h, w, t, "f32")
    w[3] = -1000.0
    same, _ = forward(h, w, t, "f32")
    assert torch.isfinite(loss).all() and torch.allclose(loss, same, rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("n,vocab,dim,dtype,grad", [
    (40, 300, 4100, "bf16", "bf16"), (40, 5000, 4096, "bf16", "f32"), (9, 1, 8192, "bf16", "bf16"), (130, 2049, 3000, "bf16", "f32"),
    (387, 260, 2050, "f32", "bf16"), (70, 4097, 1100, "f32", "f32"), (200, 129, 5000, "f32", "f32"),
    (5, 300, 4100, "f32", "f32"), (40, 700, 2050, "f32", "bf16"), (64, 129, 1537, "f32", "f32"), (23, 33, 8191, "f32", "bf16"),
    (3000, 97, 130, "bf16", "bf16"), (5001, 65, 64, "bf16", "f32"), (1371, 450, 203, "f32", "f32"), (2000, 40, 301, "f32", "bf16")])
def test_few_tiles_of_long_sums(n, vocab, dim, dtype, grad):
    """Fewer tiles than CUs: the sums of the logits, or of the head's gradient, are in parts."""
    g = gen(dim)
    w, h = matrix(g, vocab, dim, dtype, 0, dim ** -0.5)[1], matrix(g, n, dim, dtype)[1]
    t = labels_of(g, n, vocab, torch.int32, 0.2)
    t[: 3] = vocab - 1
    loss, lse = forward(h, w, t, dtype)
    check_forward(h, w, t, loss, lse)
    c = torch.rand(n, generator=g, device="cuda") + 0.5
    for first in (False, True):
        flat, old = matrix(g, vocab, dim, grad, 3)
        if first:
            old[:] = float("nan")
        dh, dw, kept = torch.full_like(h, float("nan")), old, old.clone()
        big, ws = scratch(n, vocab, dim, dtype, grad)
        zs.zs_linear_cross_entropy_backward(h, w, t, lse, dh, dw, dloss=c, scale=0.5, first=first, workspace=ws)
        assert (big[ws.numel():] == 0xFF).all()
        assert torch.isnan(flat[:vocab * (dim + 3)].view(vocab, dim + 3)[:, dim:]).all()
        check_backward(h, w, t, lse, 0.5 * f64(c), dh, dw, kept, first)
