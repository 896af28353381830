"""Pins of the generator, MXFP4, rotary and dropout oracles: published vectors, closed forms, brute
force and differences, none of them through the functions under test."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import dropout as DO
from oracle import floats as F
from oracle import mxfp4 as MX
from oracle import philox as PH
from oracle import rotary as RO


def test_philox_known_answers():
    """The vectors published with the generator (zeros, ones, and digits of pi)."""
    ones = 0xFFFFFFFF
    for key, ctr, want in (
            ((0, 0), (0, 0, 0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones, ones), (ones,) * 4, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0xA4093822, 0x299F31D0), (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert PH.philox_one(key, ctr) == want


def test_philox_arrays_equal_integers():
    seed, off = 0xA4093822299F31D0, 0x0370734413198A2E
    w = PH.philox(seed, off, np.arange(5, dtype=np.uint64)[None, :] | np.uint64(2 << 30),
                  np.array([0, 7, 2 ** 32 - 1], np.uint64)[:, None])
    for i, row in enumerate((0, 7, 2 ** 32 - 1)):
        for g in range(5):
            want = PH.philox_one((seed % 2 ** 32, seed >> 32), (g | 2 << 30, row, off % 2 ** 32, off >> 32))
            assert tuple(int(v) for v in w[i, g]) == want


def test_draws_take_bits_low_first():
    w = PH.philox(5, 9, np.uint64(3), np.uint64(1))
    d8, d16 = PH.draws(5, 9, 2, 64, 8, 0), PH.draws(5, 9, 2, 32, 16, 0)
    for b in range(16):
        assert d8[1, 48 + b] == (int(w[b // 4]) >> (8 * (b % 4))) & 0xFF
    for b in range(8):
        assert d16[1, 24 + b] == (int(w[b // 2]) >> (16 * (b % 2))) & 0xFFFF


@pytest.mark.parametrize("stochastic", [False, True])
def test_scale_exponent_by_rationals(stochastic):
    for num in (1, 3, 5, 6, 7, 11, 12, 13, 97):
        for k in (-130, -127, -3, 0, 4, 100):
            amax = Fraction(num) * Fraction(2) ** k
            e = -400
            if stochastic:
                while amax > 6 * Fraction(2) ** e:
                    e += 1
            else:
                while Fraction(2) ** (e + 3) <= amax:     # 2^(e + 2) <= amax < 2^(e + 3)
                    e += 1
            assert MX.scale_exponent(float(amax), stochastic) == max(e, -127)
    assert MX.scale_exponent(0.0, stochastic) == -127


def test_stochastic_codes_by_rationals_and_mean():
    """Every byte r at a spread of y: up exactly when the fraction says so, and the mean over r is y to
    1/512 of a step."""
    grid = [Fraction(v) for v in (0, .5, 1, 1.5, 2, 3, 4, 6)]
    r = np.arange(256)
    for y in [0.0, 2.0 ** -20, 0.1, 0.25, 0.499, 0.5, 0.75, 1.0, 1.3, 1.999, 2.0, 2.5, 3.0, 3.75, 4.0, 5.0, 5.999, 6.0]:
        y = float(np.float32(y))
        got = MX.codes_stochastic(np.full(256, y), np.zeros(256, bool), r)
        fy = Fraction(y) if y >= 1 else Fraction(round(Fraction(y) * 2 ** 23), 2 ** 23)
        low = max(i for i, v in enumerate(grid) if v <= fy)
        if low == 7:
            assert np.all(got == 7)
            continue
        step = grid[low + 1] - grid[low]
        want = [low + ((fy - grid[low]) / step + Fraction(2 * k + 1, 512) >= 1) for k in range(256)]
        assert got.tolist() == want
        mean = np.mean([float(grid[c]) for c in got])
        assert abs(mean - y) <= float(step) / 512 + 1e-7


def test_nearest_error_bound_and_special_blocks():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((6, 100)) * np.exp2(rng.integers(-20, 20, (6, 1)))).astype(np.float32)
    x[0, 40] = np.nan
    x[1, 3] = -np.inf
    x[2, 64:96] = 0
    p, s = MX.quantize_rowwise(x)
    assert p.shape == (6, 64) and s.shape == (6, 4)
    assert s[0, 1] == 0xFF and not p[0, 16:32].any() and s[1, 0] == 0xFF and s[2, 2] == 0
    v = MX.dequantize(p, s, 100)
    assert np.isnan(v[0, 32:64]).all() and np.isnan(v[1, :32]).all() and np.all(v[2, 64:96] == 0)
    amax = np.max(np.abs(np.where(np.isfinite(x), x, 0)).reshape(6, -1)[:, :96].reshape(6, 3, 32), axis=2)
    for i in range(2, 6):
        for b in range(3):
            err = np.abs(v[i, 32 * b:32 * b + 32] - x[i, 32 * b:32 * b + 32])
            assert np.all(err <= amax[i, b] / 4)       # half of the widest step (2 of 8), or the clip of [6, 8)
    # the low nibble is the even element, and the padding is zero
    one = np.zeros((1, 33), np.float32)
    one[0, 0], one[0, 1], one[0, 32] = 6.0, -0.5, 1.0
    p, s = MX.quantize_rowwise(one)
    assert p[0, 0] == 0x7 | (0x9 << 4) and s[0, 0] == 127 and s[0, 1] == 125 and p[0, 16] == 0x6 and not p[0, 17:].any()


def test_columnwise_is_rowwise_of_the_transpose():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((70, 45)).astype(np.float32)
    p, s = MX.quantize_columnwise(x)
    for c in (0, 17, 44):
        q, t = MX.quantize_rowwise(np.ascontiguousarray(x[:, c:c + 1].T))
        assert np.array_equal(p[c:c + 1], q) and np.array_equal(s[c:c + 1], t)
    a, _ = MX.quantize_columnwise(x, rng=(3, 4))
    b, _ = MX.quantize_rowwise(np.ascontiguousarray(x.T), rng=(3, 4))
    assert not np.array_equal(a, b)                    # another stream of the generator


def test_rotation_by_hand_norms_and_inverse():
    x = np.array([[[1.0, 0.0, 0.0, 2.0, 9.0]]])
    quarter = [2 ** 62, 2 ** 61]                        # a quarter and an eighth of a turn a position
    y = RO.rotate(x, [1], quarter, interleaved=False)
    c = math.sqrt(0.5)
    assert np.allclose(y, [[[0.0, -2 * c, 1.0, 2 * c, 9.0]]], atol=1e-15)
    y = RO.rotate(x, [3], quarter, interleaved=True)    # three quarters; three eighths
    assert np.allclose(y, [[[0.0, -1.0, -2 * c, -2 * c, 9.0]]], atol=1e-15)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((7, 3, 8))
    f, _ = RO.frequencies(6)
    t = [round(v / (2 * math.pi) * 2 ** 64) for v in f]
    pos = [0, 1, -5, 2 ** 31 - 1, -2 ** 40, 131072, 77]
    for il in (False, True):
        y = RO.rotate(x, pos, t, il, 1.5)
        assert np.allclose(np.linalg.norm(y[..., :6], axis=-1), 1.5 * np.linalg.norm(x[..., :6], axis=-1))
        assert np.allclose(RO.rotate(y, pos, t, il, 1 / 1.5, inverse=True), x)
        # the gradient of <g, rotate(x)> is the inverse rotation of g, by differences
        g = rng.standard_normal(x.shape)
        dx = RO.rotate(g, pos, t, il, 1.5, inverse=True)
        h = np.zeros_like(x)
        h[4, 1, 3] = 1e-6
        diff = (np.sum(g * RO.rotate(x + h, pos, t, il, 1.5)) - np.sum(g * RO.rotate(x - h, pos, t, il, 1.5))) / 2e-6
        assert abs(diff - dx[4, 1, 3]) < 1e-8


def test_scalings():
    f, s = RO.frequencies(64, 500000.0, "bands", 32.0, 1.0, 4.0, 8192)
    g, _ = RO.frequencies(64, 500000.0)
    turns = 8192 * g / (2 * math.pi)
    assert s == 1.0 and np.all(f[turns >= 4] == g[turns >= 4]) and np.allclose(f[turns <= 1] * 32, g[turns <= 1])
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and np.all((f[mid] < g[mid]) & (f[mid] * 32 > g[mid]))
    f, s = RO.frequencies(64, 10000.0, "ramp", 4.0, 1.0, 32.0, 4096)
    g, _ = RO.frequencies(64, 10000.0)
    assert f[0] == g[0] and abs(f[-1] * 4 - g[-1]) < 1e-18 and abs(s - (0.1 * math.log(4) + 1)) < 1e-15
    f, _ = RO.frequencies(64, 10000.0, "base", 4.0)
    assert f[0] == 1.0 and abs(f[-1] * 4 / g[-1] - 1) < 1e-12   # the slowest pair is stretched by the factor


def test_dropout_by_loops_gradient_and_mean():
    x = np.arange(1.0, 41.0).reshape(2, 20)
    rng = (11, 2 ** 40 + 5)
    out = DO.dropout(x, 0.25, rng, residual=np.full((2, 20), 100.0))
    for i in range(2):
        for j in range(20):
            w = PH.philox_one((11, 0), (j // 8, i, 5, 2 ** 8))
            kept = ((w[(j % 8) // 2] >> (16 * (j % 2))) & 0xFFFF) >= 16384
            assert out[i, j] == 100 + (x[i, j] * (65536 / 49152) if kept else 0)
    g = np.random.default_rng(0).standard_normal(x.shape)
    dx = DO.dropout(g, 0.25, rng)
    for i, j in ((0, 0), (1, 13), (1, 19)):
        h = np.zeros_like(x)
        h[i, j] = 0.5                                   # the map is linear: differences are exact to rounding
        d = np.sum(g * DO.dropout(x + h, 0.25, rng)) - np.sum(g * DO.dropout(x - h, 0.25, rng))
        assert abs(d - dx[i, j]) < 1e-9
    n = 400000
    kept = DO.keep((1, 2), 400, 1000, 0.1).mean()
    assert abs(kept - (1 - 6554 / 65536)) < 5 * math.sqrt(0.09 / n)
    assert not DO.keep((1, 2), 5, 5, 1.0).any() and DO.keep((1, 2), 5, 5, 0.0).all()
    bad = np.array([[np.nan, np.inf] * 8])
    assert np.all(DO.dropout(bad, 1.0, (0, 0)) == 0)


def test_values_are_exact_in_bf16():
    """Every value below 2^128 is a bf16 number; byte 253 under codes of 4 and 6 passes the type's range (and reads
    as Inf there), which takes an amax above 1.5 * 2^127 and a stochastic round up."""
    p = np.arange(256, dtype=np.uint8)[None, :].repeat(3, 0)[:, :256]
    s = np.broadcast_to(np.array([0, 1, 60, 127, 200, 250, 253, 2] * 2, np.uint8), (3, 16))
    v = MX.dequantize(p, s, 512)
    want = np.where(np.abs(v) < 2.0 ** 128, v, np.copysign(np.inf, v))
    assert np.array_equal(F.bf16_bits_to_f64(F.f64_to_bf16_bits(v)), want)
