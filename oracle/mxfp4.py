"""MXFP4 quantize and the three products on MXFP4 views (oracle; test infrastructure).

OCP Microscaling (MX) v1.0 MXFP4: E2M1 elements, one E8M0 scale per block of 32, the same blocks as
[GTP] §1.3's MXFP8 weights.  A row is zero-padded to whole blocks.  Scales as exponents e, byte e + 127,
clamped at byte 0:
  nearest     e = floor(log2 amax) - 2, code = RNE_E2M1(x / 2^e) saturated at 6
  stochastic  the least e with amax <= 6 * 2^e; y = |x| / 2^e (23 fractional bits below 1), low the grid
              point below, s the step there: up iff (y - low) / s + (2 r + 1) / 512 >= 1
A block holding NaN or Inf: byte 0xFF, codes 0.  All in exact rational or float64 arithmetic.
"""
from __future__ import annotations

import numpy as np

from . import philox as PH
from .floats import bf16_bits_to_f32, e2m1_decode, e2m1_rne_satfinite
from .sf_layout import tile_scales, untile_scales

BLOCK = 32
SCALE_NAN = 0xFF
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _as_f32(x, bf16_bits):
    return bf16_bits_to_f32(x) if bf16_bits else np.asarray(x, dtype=np.float32)


def scale_exponent(amax, stochastic: bool) -> np.ndarray:
    """e from a float64 amax (finite): by logarithm of the exact value, not its encoding."""
    amax = np.asarray(amax, np.float64)
    m, e = np.frexp(amax)                      # amax = m 2^e, 0.5 <= m < 1
    e = e - 1 - 2                              # floor(log2 amax) - 2
    if stochastic:
        e = np.where(np.ldexp(6.0, e) < amax, e + 1, e)
    return np.maximum(np.where(amax == 0, -127, e), -127)


def codes_stochastic(y, sign, r) -> np.ndarray:
    """E2M1 codes of magnitudes y in [0, 6] (float64) with random bytes r."""
    y = np.where(y < 1, np.rint(y * 2.0 ** 23) * 2.0 ** -23, y)
    low = np.searchsorted(GRID, y, side="right") - 1
    step = np.where(y < 2, 0.5, np.where(y < 4, 1.0, 2.0))
    up = (y - GRID[low]) / step + (2 * r + 1) / 512.0 >= 1.0
    return (low + up + 8 * sign).astype(np.uint8)


def quantize_rowwise(x, bf16_bits: bool = False, rng=None, stream: int = PH.ROUND_ROW):
    """[R, C] -> (packed uint8 [R, 16 ceil(C/32)], scale bytes [R, ceil(C/32)]); rng = (seed, offset)."""
    x = _as_f32(x, bf16_bits)
    R, C = x.shape
    B = -(-C // BLOCK)
    pad = np.zeros((R, B * BLOCK), np.float32)
    pad[:, :C] = x
    xb = pad.reshape(R, B, BLOCK).astype(np.float64)
    finite = np.all(np.isfinite(xb), axis=2)
    xb = np.where(finite[:, :, None], xb, 0.0)
    e = scale_exponent(np.max(np.abs(xb), axis=2), rng is not None)
    q = np.ldexp(xb, -e[:, :, None])
    if rng is None:
        codes = e2m1_rne_satfinite(q).astype(np.uint8)
    else:
        r = PH.draws(rng[0], rng[1], R, B * BLOCK, 8, stream).reshape(R, B, BLOCK)
        codes = codes_stochastic(np.abs(q), np.signbit(xb), r)
    codes = np.where(finite[:, :, None], codes, 0).astype(np.uint8).reshape(R, B * BLOCK)
    scales = np.where(finite, e + 127, SCALE_NAN).astype(np.uint8)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), scales


def quantize_columnwise(x, bf16_bits: bool = False, rng=None):
    """The rowwise view of x^T, with the columnwise rounding stream."""
    return quantize_rowwise(np.ascontiguousarray(np.asarray(x).T), bf16_bits, rng, PH.ROUND_COL)


def view(packed, scales):
    """(packed, tiled scales): the form the library writes and reads."""
    return packed, tile_scales(scales)


def dequantize(packed, scales, cols: int) -> np.ndarray:
    """float64 [R, cols] values of a view with scale bytes [R, blocks]."""
    R = packed.shape[0]
    codes = np.empty((R, packed.shape[1] * 2), np.uint8)
    codes[:, 0::2], codes[:, 1::2] = packed & 0xF, packed >> 4
    v = np.ldexp(e2m1_decode(codes).reshape(R, -1, BLOCK), scales.astype(np.int64)[:, :, None] - 127)
    v = np.where((scales == SCALE_NAN)[:, :, None], np.nan, v)
    return v.reshape(R, -1)[:, :cols]


def dequantize_tiled(packed, tiled, cols: int) -> np.ndarray:
    return dequantize(packed, untile_scales(tiled, packed.shape[0], -(-cols // BLOCK)), cols)
