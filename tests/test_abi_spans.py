"""Row strides that are each within range but carry the last row past any memory (and past 64 bits of bytes) are refused on
the host, before anything is launched.  Fake addresses."""
import ctypes as C

import pytest

from param_buffers_gb300 import abi

pytestmark = pytest.mark.skipif(not abi.LIB_PATH.exists(), reason="libgtp.so not built")
A = [0x100000 + k * (1 << 24) for k in range(5)]
ROWS, WIDE = 1 << 24, 1 << 40                # 2^64 elements from the first row to the last


def test_dropout_spans():
    lib, rng = abi.load(), C.byref(abi.gtp_rng(1, 2))

    def d(xl=64, rl=64, ol=64, res=A[1], fn=lib.gtp_dropout_add):
        return fn(A[0], abi.GTP_BF16, xl, res, rl, A[2], abi.GTP_F32, ol, ROWS, 64, 0.1, rng, None)
    assert d(xl=WIDE) == d(rl=WIDE) == d(ol=WIDE) == abi.GTP_E_SHAPE
    for xl, ol in ((WIDE, 64), (64, WIDE)):
        assert lib.gtp_dropout_grad(A[0], abi.GTP_BF16, xl, A[2], abi.GTP_BF16, ol, ROWS, 64, 0.1, rng, None) \
            == abi.GTP_E_SHAPE


def test_quantize_spans():
    lib = abi.load()
    for dt in (abi.GTP_F32, abi.GTP_BF16):
        assert lib.gtp_mxfp4_quantize(A[0], dt, ROWS, 64, WIDE, A[1], A[2], None, None, None, None) == abi.GTP_E_SHAPE
