"""Arguments of the rotary binding that do not fit the descriptor's fields are refused in words (host only)."""
import pytest
import torch

import param_buffers_gb300 as gtp


class Device:
    """A stand-in for a CUDA tensor; nothing reads its memory."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.mark.parametrize("bad", [dict(pos0=0.5), dict(pos0="7"), dict(pos0=1 << 63), dict(tokens_per_position=1.0),
                                 dict(positions_per_sequence=-(1 << 70)), dict(scale="1")])
def test_numbers_that_do_not_fit_are_value_errors(bad, monkeypatch):
    monkeypatch.setitem(gtp._TORCH_DTYPES, torch.float32, gtp._F32)
    h = Device(torch.empty(5, 3, 64, device="meta"))
    with pytest.raises(ValueError, match="64-bit"):
        gtp.gtp_rotary(h, h, [1] * 32, **bad)
