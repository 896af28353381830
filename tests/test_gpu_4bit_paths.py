"""Paths of the 4-bit step's kernels that the sizes of their other tests do not take: fp32 rows on 16 bytes but not on
32, and calls that go out as several launches (more than 2^30 groups)."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import dropout as DO
from oracle import mxfp4 as MX
from oracle import philox as PH
from oracle.sf_layout import tile_scales

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rng", [None, (17, 9)], ids=["nearest", "stochastic"])
@pytest.mark.parametrize("R,C,ld,shift", [(130, 204, 204, 0),      # a stride of 51 vectors of 16 bytes
                                          (257, 256, 264, 4),      # a base 16 bytes past 32
                                          (129, 128, 132, 4), (3, 36, 36, 0)])
def test_fp32_rows_on_16_bytes(R, C, ld, shift, rng):
    x = np.random.default_rng(R).standard_normal((R, C)).astype(np.float32)
    x[R // 2, C // 2], x[0, C - 1] = np.nan, 0.0
    store = torch.full((R * ld + shift + 8,), 7.0, device=DEV)
    src = store.as_strided((R, C), (ld, 1), shift)
    src.copy_(torch.from_numpy(x))
    assert src.data_ptr() % 16 == 0 and (src.data_ptr() % 32 or 4 * ld % 32)
    for row_only, col_only in ((0, 0), (1, 0), (0, 1)):
        row, col = gtp.gtp_mxfp4_views(R, C, DEV)
        gtp.gtp_mxfp4_quantize(src, row=None if col_only else row, col=None if row_only else col, rng=rng)
        for got, (codes, scales), skip in ((row, MX.quantize_rowwise(x, rng=rng), col_only),
                                           (col, MX.quantize_columnwise(x, rng=rng), row_only)):
            if not skip:
                assert np.array_equal(got[0].cpu().numpy(), codes)
                assert np.array_equal(got[1].cpu().numpy(), tile_scales(scales))


ROWS = (1 << 29) + 200        # two groups a row: the second launch starts at row 2^29
SAMPLE = [0, 1, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, ROWS - 1]


@pytest.mark.parametrize("C", [17, 32])
def test_values_of_several_launches(C):
    codes = torch.empty(ROWS, 16, dtype=torch.uint8, device=DEV).random_(0, 256)
    scales = torch.empty(-(-ROWS // 128) * 512, dtype=torch.uint8, device=DEV).random_(100, 150)
    out = torch.full((ROWS, C), float("nan"), dtype=torch.bfloat16, device=DEV)
    gtp.gtp_mxfp4_dequantize(codes, scales, out)
    r = torch.tensor(SAMPLE, device=DEV)
    byte = scales[(r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4]
    want = MX.dequantize(codes[r].cpu().numpy(), byte.cpu().numpy()[:, None], C)
    assert np.array_equal(out[r].double().cpu().numpy(), want)
    assert not torch.isnan(out[::1 << 20]).any() and not torch.isnan(out[-300:]).any()


@pytest.mark.parametrize("shift", [0, 1], ids=["alike", "lying differently"])
def test_dropout_of_several_launches(shift):
    C, p, rng = 9, 0.25, (3, 1 << 40)
    store = torch.empty(ROWS * C + shift, dtype=torch.bfloat16, device=DEV).fill_(1.0)
    x = store[shift:].view(ROWS, C)
    out = torch.full((ROWS, C), float("nan"), dtype=torch.bfloat16, device=DEV)
    gtp.gtp_dropout_add(x, None, out, p, rng)
    w = PH.philox(*rng, np.arange(2, dtype=np.uint64)[None, :], np.array(SAMPLE, np.uint64)[:, None])
    keep = w.astype("<u4").view("<u2").reshape(len(SAMPLE), -1)[:, :C] >= DO.threshold(p)
    got = out[torch.tensor(SAMPLE, device=DEV)].double().cpu().numpy()
    scale = 65536 / (65536 - DO.threshold(p))          # 4/3; the product is rounded to fp32, then to bf16
    assert np.array_equal(got != 0, keep)
    assert np.all(np.abs(got - scale)[keep] <= (2.0 ** -23 + 2.0 ** -8) * scale)
    assert not torch.isnan(out[::1 << 20]).any() and not torch.isnan(out[-300:]).any()
