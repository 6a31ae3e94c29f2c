"""Root-mean-square norm with the residual's addition, and its gradients
(oracle; test infrastructure only).

  h = x + r,  rstd = 1 / sqrt(sum(h^2) / D + eps),  y = h rstd w
  xh = h rstd,  dh = rstd (dy w - xh mean_D(dy w xh)) + dres,  dw = sum_rows dy xh

Everything in fp64. Where w, r or dres is None it is one or zero.
"""
from __future__ import annotations

import numpy as np


def rms_norm_forward(x, w=None, r=None, eps=1e-5):
    """(y, h, rstd)."""
    h = np.asarray(x, np.float64)
    if r is not None:
        h = h + np.asarray(r, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return (y if w is None else y * np.asarray(w, np.float64)), h, rstd


def rms_norm_backward(dy, h, w, rstd, dres=None):
    """(dh, dw) for the statistics as given."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = h * rstd
    g = dy if w is None else dy * np.asarray(w, np.float64)
    dh = rstd * (g - xh * (g * xh).mean(1, keepdims=True))
    return (dh if dres is None else dh + np.asarray(dres, np.float64)), (dy * xh).sum(0)
