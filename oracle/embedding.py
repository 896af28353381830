"""The token embedding of a vocabulary shard and its gradient (oracle; test infrastructure): float64, token by token."""
from __future__ import annotations

import numpy as np


def lookup(ids, table, first_row: int, scale: float) -> np.ndarray:
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        r = int(i) - first_row
        if 0 <= r < len(table):
            out[t] = scale * table[r]
    return out


def gradient(ids, dout, rows: int, first_row: int, scale: float):
    """(grad, sums of magnitudes, tokens) of each row of the shard."""
    dout = np.asarray(dout, np.float64)
    grad, mass, n = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1])), np.zeros(rows, np.int64)
    for t, i in enumerate(ids):
        r = int(i) - first_row
        if 0 <= r < rows:
            grad[r] += scale * dout[t]
            mass[r] += np.abs(scale * dout[t])
            n[r] += 1
    return grad, mass, n
