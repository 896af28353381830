"""Dropout with the residual add, and its gradient (oracle; test infrastructure): float64.

keep(i, j) = r >= T, r 16 bits of the generator, T = round(65536 p) (ties to even); kept elements are
scaled by 65536 / (65536 - T), dropped ones contribute 0 whatever they hold.
"""
from __future__ import annotations

import numpy as np

from . import philox as PH


def threshold(p: float) -> int:
    return int(np.rint(float(np.float32(p)) * 65536))


def keep(rng, rows: int, cols: int, p: float) -> np.ndarray:
    return PH.draws(rng[0], rng[1], rows, cols, 16, PH.DROPOUT) >= threshold(p)


def dropout(x, p: float, rng, residual=None) -> np.ndarray:
    x = np.asarray(x, np.float64)
    t = threshold(p)
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    with np.errstate(invalid="ignore"):
        out = np.where(keep(rng, *x.shape, p), x * scale, 0.0)
        return out if residual is None else np.asarray(residual, np.float64) + out
