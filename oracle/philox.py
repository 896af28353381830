"""The counter-based random numbers of stochastic rounding and dropout (oracle; test infrastructure).

Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel Random Numbers: As Easy as 1, 2, 3", SC 2011),
written with Python integers, one counter at a time, and once more on uint64 arrays.
"""
from __future__ import annotations

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
MASK = 2 ** 32 - 1
DROPOUT, ROUND_ROW, ROUND_COL = 0, 1, 2


def philox_one(key, counter):
    """The four 32-bit words of one counter, in Python integers."""
    k0, k1 = key
    x0, x1, x2, x3 = counter
    for _ in range(10):
        a, b = M0 * x0, M1 * x2
        x0, x1, x2, x3 = (b >> 32) ^ x1 ^ k0, b & MASK, (a >> 32) ^ x3 ^ k1, a & MASK
        k0, k1 = (k0 + W0) & MASK, (k1 + W1) & MASK
    return x0, x1, x2, x3


def philox(seed: int, offset: int, group, row):
    """uint32 [..., 4] words of the counters (group, row, offset) under the key seed."""
    group, row = np.broadcast_arrays(np.asarray(group, np.uint64), np.asarray(row, np.uint64))
    x = [group, row, np.full(group.shape, offset & MASK, np.uint64), np.full(group.shape, offset >> 32, np.uint64)]
    lo, s = np.uint64(MASK), np.uint64(32)
    for n in range(10):
        k0 = np.uint64(((seed & MASK) + n * W0) & MASK)
        k1 = np.uint64(((seed >> 32) + n * W1) & MASK)
        a, b = np.uint64(M0) * x[0], np.uint64(M1) * x[2]
        x = [(b >> s) ^ x[1] ^ k0, b & lo, (a >> s) ^ x[3] ^ k1, a & lo]
    return np.stack(x, -1).astype(np.uint32)


def draws(seed: int, offset: int, rows: int, cols: int, bits: int, stream: int) -> np.ndarray:
    """[rows, cols] random integers of 8 or 16 bits: 128 / bits columns a group, low bits of word 0 first."""
    per = 128 // bits
    groups = -(-cols // per)
    w = philox(seed, offset, np.arange(groups, dtype=np.uint64)[None, :] | np.uint64(stream << 30),
               np.arange(rows, dtype=np.uint64)[:, None])
    flat = np.ascontiguousarray(w.astype("<u4")).view("<u1" if bits == 8 else "<u2")
    return flat.reshape(rows, groups * per)[:, :cols].astype(np.int64)
