"""Softmax cross entropy of a large vocabulary from hidden states and the head's
weight, and its gradients (oracle; test infrastructure only).

  z = h W^T,  lse_i = log sum_v exp(z_iv),  loss_i = lse_i - z_i,label_i
  g_iv = c_i (exp(z_iv - lse_i) - [v = label_i]),  dh = g W,  dW = g^T h

Everything in fp64. Tokens whose label is outside of the vocabulary have a loss,
a log sum and gradients of zero, whatever their hidden states hold.
"""
from __future__ import annotations

import numpy as np


def counted(labels, vocab):
    labels = np.asarray(labels, np.int64)
    return (labels >= 0) & (labels < vocab)


def loss_forward(h, w, labels):
    """(loss, lse)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    labels = np.asarray(labels, np.int64)
    loss, lse = np.zeros(len(h)), np.zeros(len(h))
    at = np.flatnonzero(counted(labels, len(w)))
    z = h[at] @ w.T
    if at.size:
        top = z.max(1)
        lse[at] = top + np.log(np.exp(z - top[:, None]).sum(1))
        loss[at] = lse[at] - z[np.arange(at.size), labels[at]]
    return loss, lse


def loss_backward(h, w, labels, lse, c):
    """(dh, dW, g) for the log sums as given and the gradient c of each token's loss."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    labels = np.asarray(labels, np.int64)
    at = np.flatnonzero(counted(labels, len(w)))
    g = np.exp(h[at] @ w.T - np.asarray(lse, np.float64)[at, None])
    g[np.arange(at.size), labels[at]] -= 1.0
    g *= np.asarray(c, np.float64)[at, None]
    dh, whole = np.zeros_like(h), np.zeros((len(h), len(w)))
    dh[at], whole[at] = g @ w, g
    return dh, g.T @ h[at], whole
