"""What the binding of the 4-bit, rotary and dropout calls refuses before the library sees it (host only)."""
import pytest
import torch

import param_buffers_gb300 as gtp


class Device:
    """A stand-in for a CUDA tensor with a CPU tensor's properties; nothing reads its memory."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def dev(*shape, dtype=torch.float32):
    return Device(torch.empty(*shape, dtype=dtype, device="meta"))


def u8(*shape):
    return dev(*shape, dtype=torch.uint8)


@pytest.fixture
def plain(monkeypatch):
    """Lets the stand-ins pass the table of dtypes, which real tensors fill."""
    gtp._TORCH_DTYPES.update({torch.float32: 0, torch.bfloat16: 1, torch.uint8: 3})


def test_host_tensors_and_types_are_refused():
    x, q = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
    for call in (lambda: gtp.gtp_mxfp4_quantize(x, row=(q, q)),
                 lambda: gtp.gtp_mxfp4_dequantize(q, q, x),
                 lambda: gtp.gtp_linear_fprop_mxfp4(q, q, q, q, x),
                 lambda: gtp.gtp_rotary(x.view(4, 1, 64), x.view(4, 1, 64), [1] * 32),
                 lambda: gtp.gtp_dropout_add(x, None, x, 0.1, (1, 2)),
                 lambda: gtp.gtp_dropout_grad(x, x, 0.1, (1, 2))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for bad in ([1.0], x.numpy(), None):
        with pytest.raises((TypeError, AttributeError)):
            gtp.gtp_dropout_grad(bad, x, 0.1, (1, 2))
    with pytest.raises(TypeError):
        gtp.gtp_mxfp4_quantize(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(TypeError):
        gtp.gtp_mxfp4_quantize(torch.zeros(4, 64, dtype=torch.int32))


def test_shapes_are_refused(plain):
    src = dev(33, 70)
    good, (cc, cs) = (u8(33, 48), u8(512)), (u8(70, 32), u8(512))
    for bad in ((u8(33, 47), u8(512)), (u8(32, 48), u8(512)), (u8(33, 48), u8(511)), (u8(33, 48), u8(1024))):
        with pytest.raises(ValueError):
            gtp.gtp_mxfp4_quantize(src, row=bad)
    with pytest.raises(ValueError):
        gtp.gtp_mxfp4_quantize(src, col=good)                         # the other view's shape
    with pytest.raises(TypeError):
        gtp.gtp_mxfp4_quantize(src, row=(dev(33, 48), u8(512)))
    with pytest.raises(ValueError):
        gtp.gtp_mxfp4_quantize(dev(2, 3, 4), row=good)
    with pytest.raises(ValueError):
        gtp.gtp_mxfp4_quantize(Device(torch.empty(70, 33, device="meta").t()), row=good)
    with pytest.raises(ValueError):
        gtp.gtp_mxfp4_quantize(src, row=good, rng=(1 << 64, 0))
    with pytest.raises(ValueError):
        gtp.gtp_mxfp4_dequantize(*good, dev(33, 97))
    with pytest.raises(ValueError):
        gtp.gtp_linear_fprop_mxfp4(*good, u8(8, 32), u8(512), dev(33, 8, dtype=torch.bfloat16))   # contractions differ
    with pytest.raises(TypeError):
        gtp.gtp_linear_fprop_mxfp4(*good, u8(8, 48), u8(512), dev(33, 8))                          # an fp32 output
    with pytest.raises(ValueError):
        gtp.gtp_linear_dgrad_mxfp4(*good, u8(8, 48), u8(512), dev(8, 33, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        gtp.gtp_linear_wgrad_accum_mxfp4(*good, u8(8, 48), u8(512), dev(264, dtype=torch.bfloat16), 0)


def test_rotary_and_dropout_arguments_are_refused(plain):
    h = dev(5, 3, 64)
    for kw in (dict(layout="quarter"), dict(positions=dev(5)), ):
        with pytest.raises((TypeError, ValueError)):
            gtp.gtp_rotary(h, h, [1] * 32, **kw)
    with pytest.raises(ValueError):
        gtp.gtp_rotary(h, dev(5, 3, 32), [1] * 32)
    with pytest.raises(ValueError):
        gtp.gtp_rotary(h, dev(5, 3, 64, dtype=torch.bfloat16), [1] * 32)
    with pytest.raises(ValueError):
        gtp.gtp_rotary(dev(5, 64), dev(5, 64), [1] * 32)
    with pytest.raises(ValueError):
        gtp.gtp_rotary(h, h, [1] * 32, positions=Device(torch.empty(4, dtype=torch.int64, device="meta")))
    with pytest.raises(OverflowError):
        gtp.gtp_rotary(h, h, [-1] * 32)
    x = dev(4, 8)
    with pytest.raises(ValueError):
        gtp.gtp_dropout_add(x, None, dev(4, 9), 0.1, (1, 2))
    with pytest.raises(ValueError):
        gtp.gtp_dropout_add(x, dev(4, 8, dtype=torch.bfloat16), dev(4, 8), 0.1, (1, 2))
    with pytest.raises(ValueError):
        gtp.gtp_dropout_grad(x, dev(8, 4), 0.1, (1, 2))
    with pytest.raises(ValueError):
        gtp.gtp_dropout_grad(x, x, 0.1, (-1, 2))
    with pytest.raises(TypeError):
        gtp.gtp_dropout_grad(x, x, 0.1, (1, 2, torch.zeros(1, dtype=torch.int64)))   # an offset on the host
    for name in ("unscaled ", "ntk"):
        with pytest.raises(ValueError):
            gtp.gtp_rotary_turns(gtp.RotaryConfig(64, scaling=name))
    with pytest.raises(gtp.GtpError):
        gtp.gtp_rotary_turns(gtp.RotaryConfig(63))
