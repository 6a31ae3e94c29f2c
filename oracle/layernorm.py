"""Layer norm's forward and backward pass (oracle; test infrastructure only).

  mean = sum(x) / D,  rstd = 1 / sqrt(sum((x - mean)^2) / D + eps),  xh = (x - mean) rstd
  y = xh w + b
  dx = rstd (dy w - mean_D(dy w) - xh mean_D(dy w xh)),  dw = sum_rows dy xh,  db = sum_rows dy

Everything in fp64. Where w or b is None it is one or zero.
"""
from __future__ import annotations

import numpy as np


def layer_norm_forward(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd):
    """(dx, dw, db) for the statistics as given."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * rstd
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
