"""Embedding lookup with scaling and its gradient (oracle; test infrastructure only).

  forward   out_i = scale table[t_i] (+ pos_table[p_i]); an id outside of its
            table selects a row of zeros
  backward  grad_v = old_v + scale sum over i with t_i = v of dout_i; ids outside
            of the table and the padding id contribute nothing

Everything in fp64 on fp64 inputs, one row at a time.
"""
from __future__ import annotations

import numpy as np


def _rows(table: np.ndarray, ids) -> np.ndarray:
    out = np.zeros((len(ids), table.shape[1]))
    for i, t in enumerate(ids):
        if 0 <= t < table.shape[0]:
            out[i] = table[t]
    return out


def embed_forward(table, tokens, scale=1.0, pos_table=None, positions=None) -> np.ndarray:
    out = _rows(np.asarray(table, np.float64), tokens) * float(scale)
    if pos_table is not None:
        out += _rows(np.asarray(pos_table, np.float64), positions)
    return out


def embed_backward(dout, tokens, vocab, scale=1.0, padding_idx=-1, old=None):
    """(grad, magnitude): magnitude is |old| + |scale| sum |dout|, what rounding errors of a sum scale with."""
    dout = np.asarray(dout, np.float64)
    grad = np.zeros((vocab, dout.shape[1]))
    size = np.zeros_like(grad)
    for i, t in enumerate(tokens):
        if 0 <= t < vocab and t != padding_idx:
            grad[t] += dout[i]
            size[t] += np.abs(dout[i])
    grad *= float(scale)
    size *= abs(float(scale))
    if old is not None:
        grad += np.asarray(old, np.float64)
        size += np.abs(np.asarray(old, np.float64))
    return grad, size
