"""Root-mean-square norm and its gradient (oracle; test infrastructure): float64, from the definitions.

forward: rstd = 1 / sqrt(mean s^2 + eps), y = s rstd w.  gradient: the Jacobian of y in s applied to dy, row by row,
  dx = rstd w dy - s rstd^3 / C * sum(s w dy) + dsum,   dw = sum over rows of dy s rstd.
"""
from __future__ import annotations

import numpy as np


def forward(s, w, eps: float):
    s, w = np.asarray(s, np.float64), np.asarray(w, np.float64)
    rstd = 1 / np.sqrt((s * s).mean(1) + eps)
    return rstd, s * rstd[:, None] * w


def gradient(dy, s, rstd, w, dsum=None):
    dy, s, rstd, w = (np.asarray(a, np.float64) for a in (dy, s, rstd, w))
    r = rstd[:, None]
    dx = r * w * dy - s * r ** 3 / s.shape[1] * (s * w * dy).sum(1, keepdims=True)
    return dx if dsum is None else dx + np.asarray(dsum, np.float64), (dy * s * r).sum(0)
