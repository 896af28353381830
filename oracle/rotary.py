"""Rotary positions (oracle; test infrastructure): float64, complex multiplication by e^{i p f}.

The whole turns of p f are removed in Python integers from the 64-bit fraction, so the float64 angle is
exact to 2^-53 of a turn at any position.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot_dim, base=10000.0, scaling="unscaled", factor=1.0, low_turns=1.0, high_turns=4.0, context=8192):
    """(frequencies in radians per position, scale of the rotated values).  "linear": position interpolation (Chen et al.
    2023); "base", "bands" and "ramp": the NTK-aware base, NTK-by-parts and YaRN (Peng et al. 2023), the last as its
    authors released it."""
    i = np.arange(rot_dim // 2, dtype=np.float64)
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":
        keep = np.clip((context * f / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0, 1)
        return keep * f + (1 - keep) * f / factor, 1.0
    if scaling == "ramp":
        def index(n):
            return rot_dim * math.log(context / (n * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(0, math.floor(index(high_turns))), min(rot_dim - 1, math.ceil(index(low_turns)))
        if last <= first:
            last = first + 0.001
        keep = np.clip(1 - (i - first) / (last - first), 0, 1)
        return keep * f + (1 - keep) * f / factor, 0.1 * math.log(factor) + 1
    return f, 1.0


def rotate(x, positions, turns, interleaved: bool, scale: float = 1.0, inverse: bool = False) -> np.ndarray:
    """x float64 [T, H, D], positions ints [T], turns ints [rot_dim / 2]."""
    x = np.asarray(x, np.float64)
    half = len(turns)
    frac = np.array([[((int(p) * int(t)) % 2 ** 64) / 2.0 ** 64 for t in turns] for p in positions])
    w = scale * np.exp((-2j if inverse else 2j) * math.pi * frac)[:, None, :]
    out = x.copy()
    if interleaved:
        z = (x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2]) * w
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = z.real, z.imag
    else:
        z = (x[..., :half] + 1j * x[..., half:2 * half]) * w
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    return out
