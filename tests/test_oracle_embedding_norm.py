"""The embedding and layer norm oracle against torch's own in fp64 and against differences."""
import numpy as np
import torch
import torch.nn.functional as F

from oracle import embedding as oe
from oracle import layernorm as ol


def test_embedding_against_torch():
    rng = np.random.default_rng(1)
    table, t = rng.standard_normal((11, 5)), rng.integers(0, 11, 40)
    pos, p = rng.standard_normal((6, 5)), rng.integers(0, 6, 40)
    dout = rng.standard_normal((40, 5))
    wt = torch.tensor(table, requires_grad=True)
    wp = torch.tensor(pos, requires_grad=True)
    out = F.embedding(torch.tensor(t), wt, padding_idx=3) * 1.5 + F.embedding(torch.tensor(p), wp)
    out.backward(torch.tensor(dout))
    np.testing.assert_allclose(oe.embed_forward(table, t, 1.5, pos, p), out.detach().numpy(), rtol=0, atol=1e-14)
    got, size = oe.embed_backward(dout, t, 11, 1.5, padding_idx=3)
    np.testing.assert_allclose(got, wt.grad.numpy(), rtol=0, atol=1e-13)
    assert np.all(size >= np.abs(got) - 1e-12)
    np.testing.assert_allclose(oe.embed_backward(dout, p, 6, old=pos)[0], wp.grad.numpy() + pos, rtol=0, atol=1e-13)


def test_embedding_ids_outside_the_table():
    table = np.arange(6.0).reshape(3, 2) + 1
    out = oe.embed_forward(table, [-1, 0, 3, 2, -100], 2.0)
    np.testing.assert_array_equal(out, [[0, 0], [2, 4], [0, 0], [10, 12], [0, 0]])
    g, _ = oe.embed_backward(np.ones((5, 2)), [-1, 0, 3, 2, 2], 3)
    np.testing.assert_array_equal(g, [[1, 1], [0, 0], [2, 2]])
    bad = np.ones((3, 2))
    bad[0] = np.nan  # the row of an ignored token reaches nothing
    assert np.isfinite(oe.embed_backward(bad, [-100, 1, 1], 3)[0]).all()


def test_layer_norm_against_torch():
    rng = np.random.default_rng(2)
    x, w, b, dy = rng.standard_normal((7, 13)) + 3, rng.standard_normal(13), rng.standard_normal(13), rng.standard_normal((7, 13))
    tx, tw, tb = (torch.tensor(a, requires_grad=True) for a in (x, w, b))
    y = F.layer_norm(tx, (13,), tw, tb, 1e-3)
    y.backward(torch.tensor(dy))
    got, mean, rstd = ol.layer_norm_forward(x, w, b, 1e-3)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=0, atol=1e-13)
    for a, t in zip(ol.layer_norm_backward(dy, x, w, mean, rstd), (tx, tw, tb)):
        np.testing.assert_allclose(a, t.grad.numpy(), rtol=0, atol=1e-12)
    plain = F.layer_norm(torch.tensor(x), (13,), None, None, 1e-3).numpy()
    np.testing.assert_allclose(ol.layer_norm_forward(x, eps=1e-3)[0], plain, rtol=0, atol=1e-13)


def test_layer_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, w, b, dy = rng.standard_normal((2, 5)), rng.standard_normal(5), rng.standard_normal(5), rng.standard_normal((2, 5))

    def loss(x, w, b):
        return float((ol.layer_norm_forward(x, w, b)[0] * dy).sum())

    _, mean, rstd = ol.layer_norm_forward(x, w, b)
    h = 1e-6
    for which, grad in enumerate(ol.layer_norm_backward(dy, x, w, mean, rstd)):
        at = [x, w, b][which]
        for i in np.ndindex(at.shape):
            args = [x.copy(), w.copy(), b.copy()]
            args[which][i] += h
            up = loss(*args)
            args[which][i] -= 2 * h
            # central differences of a smooth function of order 1: h^2 and 1e-16 / h both near 1e-10
            assert abs((up - loss(*args)) / (2 * h) - grad[i]) < 1e-7
