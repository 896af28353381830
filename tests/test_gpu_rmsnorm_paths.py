"""The norm where its kernels change: clusters of every size for the columnwise view.  Tolerances as test_gpu_rmsnorm.py
derives them."""
import pytest
import torch

import param_buffers_gb300 as gtp
from test_gpu_rmsnorm import B, DEV, F, check_forward, check_view, matrix, views

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("xd,rd", [(B, B), (F, None), (B, F), (F, B)])
@pytest.mark.parametrize("C", [224, 512, 768, 1024, 1280, 1376, 1536, 1792, 2016])
def test_clusters_of_one_to_eight(C, xd, rd):
    """Blocks of 256 columns share a row's sum of squares: one to eight of them, the last one whole or not."""
    R = 160
    x, w = matrix(R, C, xd), (1 + 0.2 * torch.randn(C, device=DEV)).to(B)
    x *= torch.exp(torch.randn(R, 1, device=DEV)).to(xd)
    res = None if rd is None else matrix(R, C, rd, 3.0)
    out = None if rd is None else torch.empty(R, C, dtype=rd, device=DEV)
    y, rstd = torch.empty(R, C, device=DEV), torch.empty(R, device=DEV)
    row, col = views(R, C, False)
    for _ in range(20):  # each over the tail of the one before
        for t in (y, rstd):
            t.fill_(float("nan"))
        gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y, rstd=rstd, row=row, col=col)
        if rd is not None:
            assert torch.equal(out, (x.float() + res.float()).to(rd))
        check_forward(x if rd is None else out, w, 1e-5, rstd, y)
    check_view(row, y, False)
    check_view(col, y.t().contiguous(), False)
