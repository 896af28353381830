"""The embedding gradient's workspace size answers -1 wherever the call refuses the sizes; a step whose rates fp32 does not hold is
refused (host only)."""
import ctypes as C

import pytest

from param_buffers_gb300 import abi

pytestmark = pytest.mark.skipif(not abi.LIB_PATH.exists(), reason="libgtp.so not built")


def call(tokens, rows, cols, bytes):
    d = abi.gtp_embedding_grad_desc(ids=1 << 45, dout=1 << 46, grad_data=1 << 47, tokens=tokens, first_row=0, rows=rows, cols=cols,
                                    dout_ld=max(cols, 1), grad_offset=0, grad_numel_total=1 << 50, scale=1.0, ids64=1,
                                    dout_dtype=abi.GTP_BF16, grad_dtype=abi.GTP_F32, reserved=0)
    return abi.load().gtp_embedding_grad_accum(C.byref(d), 1 << 48, bytes, None)


@pytest.mark.parametrize("tokens,rows,cols", [(1 << 30, 8, 2048), (8, 1 << 30, 2048), (1 << 30, 1 << 30, 1025), (1025, 8, 1 << 30),
                                              (1 << 21, 1 << 10, (1 << 19) + 1), ((1 << 30) + 1, 1, 1), (1, (1 << 30) + 1, 1), (1, 1, -1)])
def test_refused_sizes(tokens, rows, cols):
    assert call(tokens, rows, cols, 1 << 62) in (abi.GTP_E_SHAPE, abi.GTP_E_ARG)
    assert abi.load().gtp_embedding_grad_workspace_bytes(tokens, rows, cols) == -1


@pytest.mark.parametrize("tokens,rows,cols", [(1 << 30, 8, 1024), (8, 1 << 30, 1024), (1 << 30, 1 << 30, 1024), (1, 1, 1), (2561, 3, 5)])
def test_sizes_at_the_limit(tokens, rows, cols):
    need = abi.load().gtp_embedding_grad_workspace_bytes(tokens, rows, cols)
    assert need > 0 and call(tokens, rows, cols, need - 1) == abi.GTP_E_CAPACITY


def step(**h):
    """A step whose hyper-parameters pass every check but, it may be, the last; its workspace is too small."""
    p = abi.gtp_muon_hparams(lr=1e-3, momentum=0.9, weight_decay=0.1, scale=1.0, grad_factor=1.0, coefficients=(3.4445, -4.7750, 2.0315),
                             steps=5, nesterov=1, zero_grad_after=1)
    for k, v in h.items():
        setattr(p, k, v)
    at = [1 << (40 + k) for k in range(5)]
    return abi.load().gtp_muon_step(at[0], abi.GTP_F32, at[1], at[2], at[3], 64, (C.c_int64 * 1)(0), 1, 8, 8, C.byref(p), at[4], 8, None)


@pytest.mark.parametrize("h,status", [(dict(lr=1e20, scale=1e20), abi.GTP_E_ARG), (dict(lr=1e20, scale=-1e20), abi.GTP_E_ARG),
                                      (dict(lr=1e30, weight_decay=1e30), abi.GTP_E_ARG), (dict(lr=1e15, scale=1e15), abi.GTP_E_CAPACITY),
                                      (dict(lr=0.0, scale=3e38), abi.GTP_E_CAPACITY)])
def test_rates_that_fp32_does_not_hold(h, status):
    """lr scale and 1 - lr weight_decay are formed on the host: Inf there would make every weight Inf or NaN."""
    assert step(**h) == status, abi.load().gtp_last_error()
