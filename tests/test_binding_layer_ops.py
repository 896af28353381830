"""What the binding of the embedding, the norm and the orthogonalised update refuses before the library sees it (host
only)."""
import pytest
import torch

import param_buffers_gb300 as gtp

B = torch.bfloat16


class Device:
    """A stand-in for a CUDA tensor with a CPU tensor's properties; nothing reads its memory."""

    def __init__(self, t):
        self._t = t
        self.is_cuda = True

    def __getattr__(self, name):
        return getattr(self._t, name)


def dev(*shape, dtype=torch.float32):
    return Device(torch.empty(*shape, dtype=dtype, device="meta"))


def turned(*shape, dtype=torch.float32):
    return Device(torch.empty(*shape, dtype=dtype, device="meta").t())


def u8(*shape):
    return dev(*shape, dtype=torch.uint8)


@pytest.fixture(autouse=True)
def plain():
    """Lets the stand-ins pass the table of dtypes, which real tensors fill."""
    gtp._TORCH_DTYPES.update({torch.float32: 0, B: 1, torch.uint8: 3})


IDS, WS = dev(7, dtype=torch.int64), u8(1 << 16)


def test_host_tensors_are_refused():
    x, v, ids, ws = torch.zeros(32, 64), torch.zeros(64), torch.zeros(32, dtype=torch.int64), torch.zeros(1 << 16, dtype=torch.uint8)
    flat = torch.zeros(1 << 16)
    for call in (lambda: gtp.gtp_embedding(ids, x, x),
                 lambda: gtp.gtp_embedding_grad_accum(x, ids, flat, 0, 32, ws),
                 lambda: gtp.gtp_rmsnorm(x, v, 1e-5, y=x),
                 lambda: gtp.gtp_rmsnorm_grad(x, x, torch.zeros(32), v, x, flat, 0, ws),
                 lambda: gtp.gtp_mxfp8_dequantize(x.byte(), torch.zeros(32, 2, dtype=torch.uint8), x),
                 lambda: gtp.gtp_orthogonalize(x, x, ws),
                 lambda: gtp.gtp_muon_step(flat, flat, flat, None, [0], 32, 64, gtp.MuonHparams(), ws)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    # a host workspace beside device operands
    d = dev(32, 64)
    for call in (lambda: gtp.gtp_embedding_grad_accum(d, dev(32, dtype=torch.int64), dev(1 << 16), 0, 32, ws),
                 lambda: gtp.gtp_rmsnorm_grad(d, d, dev(32), dev(64), d, dev(1 << 16), 0, ws),
                 lambda: gtp.gtp_orthogonalize(d, d, ws),
                 lambda: gtp.gtp_muon_step(dev(4096), dev(4096), dev(4096), None, [0], 32, 64, gtp.MuonHparams(), ws)):
        with pytest.raises(ValueError, match="workspace"):
            call()


@pytest.mark.parametrize("error,ids,table,out,kw", [
    (TypeError, dev(7), dev(9, 8), dev(7, 8), {}),                                   # ids of floats
    (TypeError, dev(7, dtype=torch.int16), dev(9, 8), dev(7, 8), {}),
    (ValueError, dev(7, 1, dtype=torch.int64), dev(9, 8), dev(7, 8), {}),
    (ValueError, Device(torch.empty(14, dtype=torch.int64, device="meta")[::2]), dev(9, 8), dev(7, 8), {}),
    (ValueError, IDS, dev(9, 8), dev(6, 8), {}), (ValueError, IDS, dev(9, 8), dev(7, 9), {}),
    (ValueError, IDS, dev(72), dev(7, 8), {}), (ValueError, IDS, turned(8, 9), dev(7, 8), {}),
    (TypeError, IDS, dev(9, 8, dtype=torch.float64), dev(7, 8), {}), (TypeError, IDS, dev(9, 8), u8(7, 8), {}),
    (ValueError, IDS, dev(9, 8), dev(7, 8), dict(first_row=1 << 63)), (ValueError, IDS, dev(9, 8), dev(7, 8), dict(first_row=0.5)),
    (ValueError, IDS, dev(9, 8), dev(7, 8), dict(scale=1e39)), (ValueError, IDS, dev(9, 8), dev(7, 8), dict(scale="1")),
])
def test_lookup(error, ids, table, out, kw):
    with pytest.raises(error):
        gtp.gtp_embedding(ids, table, out, **kw)


@pytest.mark.parametrize("error,change", [
    (ValueError, dict(dout=dev(6, 8))), (TypeError, dict(dout=u8(7, 8))), (ValueError, dict(dout=turned(8, 7))),
    (TypeError, dict(grad_data=u8(99))), (ValueError, dict(grad_data=turned(9, 11))),
    (ValueError, dict(workspace=Device(torch.empty(99, dtype=torch.uint8, device="meta")[::2]))),
    (ValueError, dict(grad_offset=1 << 63)), (ValueError, dict(rows=2.0)), (ValueError, dict(scale=None)),
])
def test_lookup_gradient(error, change):
    a = dict(dout=dev(7, 8), ids=IDS, grad_data=dev(99), grad_offset=0, rows=9, workspace=WS)
    with pytest.raises(error):
        gtp.gtp_embedding_grad_accum(**{**a, **change})


@pytest.mark.parametrize("error,change", [
    (ValueError, dict(x=dev(64))), (ValueError, dict(x=turned(64, 32))), (TypeError, dict(x=u8(32, 64))),
    (ValueError, dict(weight=dev(63))), (ValueError, dict(weight=dev(1, 64))), (TypeError, dict(weight=u8(64))),
    (ValueError, dict(residual=dev(32, 64))), (ValueError, dict(sum=dev(32, 64))),                 # together or not at all
    (ValueError, dict(residual=dev(32, 64), sum=dev(32, 64, dtype=B))), (ValueError, dict(residual=dev(32, 63), sum=dev(32, 63))),
    (ValueError, dict(y=dev(31, 64))), (TypeError, dict(rstd=dev(32, dtype=B))), (ValueError, dict(rstd=dev(31))),
    (TypeError, dict(row=(dev(32, 64), u8(32, 2)))), (ValueError, dict(row=(u8(64, 32), u8(32, 2)))),
    (ValueError, dict(row=(u8(32, 64), u8(32, 3)))), (ValueError, dict(row=(u8(32, 64), u8(511)))),
    (ValueError, dict(row=(u8(32, 64),))), (ValueError, dict(col=(u8(32, 64), u8(64, 1)))),
    (ValueError, dict(row=(u8(32, 64), u8(32, 2)), col=(u8(64, 32), u8(512)))),                    # tiled and not
    (ValueError, dict(row=(turned(64, 32, dtype=torch.uint8), u8(32, 2)))),
    (ValueError, dict(eps=1e39)), (ValueError, dict(eps="0")),
])
def test_norm(error, change):
    a = dict(x=dev(32, 64), weight=dev(64), eps=1e-5, y=dev(32, 64), rstd=dev(32))
    with pytest.raises(error):
        gtp.gtp_rmsnorm(**{**a, **change})


@pytest.mark.parametrize("error,change", [
    (ValueError, dict(sum=dev(32, 63))), (ValueError, dict(dx=dev(31, 64))), (ValueError, dict(dx=dev(32, 64, dtype=B))),
    (ValueError, dict(dsum=dev(32, 64, dtype=B))), (ValueError, dict(dsum=dev(32, 32))), (ValueError, dict(weight=dev(32))),
    (ValueError, dict(rstd=dev(64))), (TypeError, dict(rstd=dev(32, dtype=B))), (TypeError, dict(grad_data=u8(64))),
    (ValueError, dict(grad_data=turned(8, 8))), (ValueError, dict(grad_offset=0.0)),
])
def test_norm_gradient(error, change):
    a = dict(dy=dev(32, 64), sum=dev(32, 64), rstd=dev(32), weight=dev(64), dx=dev(32, 64), grad_data=dev(64), grad_offset=0,
             workspace=WS)
    with pytest.raises(error):
        gtp.gtp_rmsnorm_grad(**{**a, **change})


def test_view_values():
    for codes, scales, out, error in ((u8(4, 64), u8(4, 2), dev(4, 32), ValueError), (u8(4, 64), u8(4, 1), dev(4, 64), ValueError),
                                      (dev(4, 64), u8(4, 2), dev(4, 64), TypeError), (u8(4, 64), u8(4, 2), turned(64, 4), ValueError),
                                      (u8(4, 64), u8(4, 2), u8(4, 64), TypeError)):
        with pytest.raises(error):
            gtp.gtp_mxfp8_dequantize(codes, scales, out)


@pytest.mark.parametrize("error,change", [
    (ValueError, dict(src=dev(8))), (ValueError, dict(src=dev(1, 2, 8, 9))), (ValueError, dict(src=turned(9, 8))),
    (TypeError, dict(src=u8(8, 9))), (TypeError, dict(out=u8(8, 9))), (ValueError, dict(out=dev(9, 8))),
    (ValueError, dict(out=dev(2, 8, 9))), (ValueError, dict(coefficients=(1.0, 2.0))), (ValueError, dict(coefficients=(1, 2, "3"))),
    (ValueError, dict(coefficients=(1e39, 0, 0))),
])
def test_orthogonalize(error, change):
    a = dict(src=dev(8, 9), out=dev(8, 9), workspace=WS)
    with pytest.raises(error):
        gtp.gtp_orthogonalize(**{**a, **change})


@pytest.mark.parametrize("error,change", [
    (TypeError, dict(grad_data=u8(99))), (TypeError, dict(momentum=dev(99, dtype=B))), (TypeError, dict(master=dev(99, dtype=B))),
    (TypeError, dict(param_data=dev(99))), (ValueError, dict(momentum=dev(98))), (ValueError, dict(master=dev(100))),
    (ValueError, dict(param_data=dev(98, dtype=B))), (TypeError, dict(grad_scale=dev(2))), (TypeError, dict(grad_scale=dev(1, dtype=B))),
    (ValueError, dict(offsets=[0.5])), (ValueError, dict(offsets=[1 << 63])),
    (ValueError, dict(h=gtp.MuonHparams(lr="1"))), (ValueError, dict(h=gtp.MuonHparams(scale=1e39))),
    (ValueError, dict(h=gtp.MuonHparams(steps=1.5))),
])
def test_step(error, change):
    a = dict(grad_data=dev(99), momentum=dev(99), master=dev(99), param_data=dev(99, dtype=B), offsets=[0], rows=8, cols=9,
             h=gtp.MuonHparams(), workspace=WS)
    with pytest.raises(error):
        gtp.gtp_muon_step(**{**a, **change})


def test_workspace_sizes_out_of_range():
    for call in (lambda: gtp.gtp_embedding_grad_workspace_bytes(-1, 1, 1), lambda: gtp.gtp_rmsnorm_grad_workspace_bytes(1, 16385),
                 lambda: gtp.gtp_orthogonalize_workspace_bytes(65, 8, 8)):
        with pytest.raises(ValueError):
            call()
