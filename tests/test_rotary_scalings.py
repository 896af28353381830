"""The context scalings of the rotary frequencies against values worked out by hand, for the oracle and for the library
(host only).  With base = 2^(rot_dim / 2), pair j has frequency 2^-j and makes 1303.8 * 2^-j turns over a context of 8192
(8192 / 2 pi = 1303.797...), so the pairs at which a number of turns is passed can be read off."""
import math

import numpy as np
import pytest

import param_buffers_gb300 as gtp
from oracle import rotary as RO
from param_buffers_gb300 import abi

FACTOR = 8.0


def of_library(rot, **kw):
    if not abi.LIB_PATH.exists():
        pytest.skip("libgtp.so not built")
    turns, scale = gtp.gtp_rotary_turns(gtp.RotaryConfig(rot, **kw))
    return np.array([t / 2.0 ** 64 * 2 * math.pi for t in turns]), scale


def of_oracle(rot, **kw):
    return RO.frequencies(rot, **kw)


def kept(rot, blend):
    """Frequencies 2^-j of which a share `blend[j]` is kept and the rest stretched by FACTOR; the pairs before the
    listed ones are kept, those after them stretched."""
    f = 2.0 ** -np.arange(rot // 2)
    b = np.array([blend.get(j, 1.0 if j < min(blend) else 0.0) for j in range(rot // 2)])
    return b * f + (1 - b) * f / FACTOR


# (rot_dim, high turns, low turns, context): the share of the unscaled frequency that a pair keeps
RAMPS = [
    # 32 turns between pairs 5 (40.7) and 6 (20.4), one between 10 (1.27) and 11 (0.64): from pair 5 to pair 11
    (64, 32.0, 1.0, 8192, {5: 1.0, 6: 5 / 6, 7: 4 / 6, 8: 3 / 6, 9: 2 / 6, 10: 1 / 6, 11: 0.0}),
    # 256 turns between pairs 2 (326) and 3 (163); the far end is held to rot_dim - 1 = 7, past the last pair
    (8, 256.0, 1.0, 8192, {2: 1.0, 3: 4 / 5}),
    # even the first pair makes 0.64 of a turn: the near end is held to 0, and both ends fall together
    (16, 2.0, 1.0, 4, {0: 1.0, 1: 0.0}),
    # 2 turns between pairs 9 and 10, one between 10 and 11
    (32, 2.0, 1.0, 8192, {9: 1.0, 10: 1 / 2, 11: 0.0}),
]


@pytest.mark.parametrize("of", [of_oracle, of_library])
@pytest.mark.parametrize("rot,high,low,context,blend", RAMPS)
def test_ramp(of, rot, high, low, context, blend):
    f, scale = of(rot, base=2.0 ** (rot // 2), scaling="ramp", factor=FACTOR, low_turns=low, high_turns=high,
                  context=context)
    assert np.allclose(f, kept(rot, blend), rtol=1e-12, atol=2.0 ** -62)   # half a unit of the library's fixed point
    assert abs(scale - (1 + 0.1 * math.log(8))) < 2.0 ** -23


@pytest.mark.parametrize("of", [of_oracle, of_library])
def test_bands(of):
    """In turns, not in pairs: 1303.797 * 2^-9 = 2.54648 and * 2^-10 = 1.27324 lie between 1 and 4."""
    f, scale = of(64, base=2.0 ** 32, scaling="bands", factor=FACTOR, low_turns=1.0, high_turns=4.0, context=8192)
    blend = {j: 1.0 for j in range(9)} | {9: (8192 / (2 * math.pi) / 512 - 1) / 3, 10: (8192 / (2 * math.pi) / 1024 - 1) / 3}
    assert abs(blend[9] - 0.515493) < 1e-6 and abs(blend[10] - 0.091080) < 1e-6
    assert np.allclose(f, kept(64, blend), rtol=1e-12, atol=2.0 ** -62) and scale == 1.0


@pytest.mark.parametrize("of", [of_oracle, of_library])
def test_linear_and_base(of):
    f, _ = of(64, base=2.0 ** 32, scaling="linear", factor=FACTOR)
    assert np.allclose(f, 2.0 ** -np.arange(32) / 8, rtol=1e-12, atol=2.0 ** -62)
    # 8^(64 / 62) times the base: pair j is stretched by 8^(j / 31), the first not at all and the last by 8
    f, _ = of(64, base=2.0 ** 32, scaling="base", factor=FACTOR)
    assert np.allclose(f, [2.0 ** -j * 8.0 ** (-j / 31) for j in range(32)], rtol=1e-12, atol=2.0 ** -62)
