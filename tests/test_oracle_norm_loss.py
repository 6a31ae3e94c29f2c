"""The RMS norm, 8-bit and loss oracle against torch's own in fp64 and against differences."""
import numpy as np
import torch
import torch.nn.functional as F

from oracle import activation as oa
from oracle import head_loss as oh
from oracle import rmsnorm as orn


def test_rms_norm_against_torch():
    rng = np.random.default_rng(1)
    x, r, w = rng.standard_normal((7, 13)), rng.standard_normal((7, 13)), rng.standard_normal(13)
    dy, dres = rng.standard_normal((7, 13)), rng.standard_normal((7, 13))
    tx, tr, tw = (torch.tensor(a, requires_grad=True) for a in (x, r, w))
    h = tx + tr
    y = F.rms_norm(h, (13,), tw, 1e-5)
    (y * torch.tensor(dy)).sum().add((h * torch.tensor(dres)).sum()).backward()
    got, gh, rstd = orn.rms_norm_forward(x, w, r, 1e-5)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=0, atol=1e-14)
    np.testing.assert_array_equal(gh, x + r)
    dh, dw = orn.rms_norm_backward(dy, gh, w, rstd, dres)
    np.testing.assert_allclose(dh, tx.grad.numpy(), rtol=0, atol=1e-14)
    np.testing.assert_allclose(dh, tr.grad.numpy(), rtol=0, atol=1e-14)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=0, atol=1e-13)


def test_codes_against_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oa.decode(codes), want)
    rng = np.random.default_rng(2)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.standard_normal(20000) * 2.0 ** -6, want[np.isfinite(want)],
                        (oa.FINITE[1:] + oa.FINITE[:-1]) / 2, [0.0, -0.0, np.nan]]).astype(np.float32)
    got = oa.encode(v.astype(np.float64))
    torch_codes = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    nan = np.isnan(v)
    np.testing.assert_array_equal(got[~nan], torch_codes[~nan])
    assert np.isnan(oa.decode(got[nan])).all()


def test_scales():
    for top, want in ((448.0, 1.0), (np.nextafter(448.0, 500), 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                      (1.76, 2.0 ** -7), (0.0, 1.0), (2.0 ** -149, 2.0 ** -117), (1.75 * 2.0 ** 127, 2.0 ** 119)):
        assert oa.scale_of(top) == want, top
    codes, scales = oa.pack(np.array([[1.0, np.inf, np.nan, -448.0, 0.0]]))
    assert scales[0, 0] == 1.0
    np.testing.assert_array_equal(oa.unpack(codes, scales), [[1.0, np.nan, np.nan, -448.0, 0.0]])
    big = oa.unpack(*oa.pack(np.full((1, 3), np.finfo(np.float32).max, np.float64)))
    np.testing.assert_array_equal(big, oa.MOST)


def test_loss_against_torch():
    rng = np.random.default_rng(3)
    h, w = rng.standard_normal((9, 6)), rng.standard_normal((11, 6))
    labels = np.array([0, 10, 3, -100, 5, 5, 11, -1, 7])
    c = rng.standard_normal(9)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    ignored = torch.tensor(np.where((labels < 0) | (labels > 10), -100, labels))
    each = F.cross_entropy(th @ tw.t(), ignored, ignore_index=-100, reduction="none")
    (each * torch.tensor(c)).sum().backward()
    loss, lse = oh.loss_forward(h, w, labels)
    np.testing.assert_allclose(loss, each.detach().numpy(), rtol=0, atol=1e-13)
    live = oh.counted(labels, 11)
    np.testing.assert_allclose(lse[live], torch.logsumexp(th @ tw.t(), 1).detach().numpy()[live], rtol=0, atol=1e-13)
    assert not lse[~live].any()
    dh, dw, g = oh.loss_backward(h, w, labels, lse, c)
    np.testing.assert_allclose(dh, th.grad.numpy(), rtol=0, atol=1e-13)
    np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=0, atol=1e-13)
    assert not dh[~live].any() and not g[~live].any()


def test_loss_against_differences():
    rng = np.random.default_rng(4)
    h, w, labels, c = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), np.array([4, -1, 0]), np.array([1.0, 2.0, -0.5])
    dh, dw, _ = oh.loss_backward(h, w, labels, oh.loss_forward(h, w, labels)[1], c)
    e = 1e-6
    for a, d in ((h, dh), (w, dw)):
        for at in np.ndindex(a.shape):
            a[at] += e
            up = (oh.loss_forward(h, w, labels)[0] * c).sum()
            a[at] -= 2 * e
            down = (oh.loss_forward(h, w, labels)[0] * c).sum()
            a[at] += e
            assert abs((up - down) / (2 * e) - d[at]) < 1e-8


def test_ignored_hidden_states_reach_nothing():
    h, w = np.ones((3, 2)), np.ones((4, 2))
    h[1] = np.nan
    labels = [0, -100, 3]
    loss, lse = oh.loss_forward(h, w, labels)
    dh, dw, _ = oh.loss_backward(h, w, labels, lse, np.ones(3))
    assert np.isfinite(loss).all() and np.isfinite(dh).all() and np.isfinite(dw).all()
