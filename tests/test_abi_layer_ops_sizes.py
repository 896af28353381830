"""The embedding gradient's workspace size answers -1 wherever the call refuses the sizes (host only)."""
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
