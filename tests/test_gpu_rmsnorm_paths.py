"""The norm where its kernels change: clusters of every size for the columnwise view, more rows than the machine has blocks
(several a thread at once, or one after the other), rows whose squares leave fp32's range on every path.  Tolerances as
test_gpu_rmsnorm.py derives them."""
import pytest
import torch

import param_buffers_gb300 as gtp
from test_gpu_rmsnorm import B, DEV, F, check_forward, check_view, forward, matrix, test_gradient as gradient, views

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


@pytest.mark.parametrize("xd,rd", [(B, None), (F, None), (B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("R,C", [(8191, 2048), (1301, 4096), (20003, 256), (5003, 520), (1303, 5120), (700, 16384), (20003, 250),
                                 (30001, 31), (20003, 1001)])
def test_more_rows_than_blocks(R, C, xd, rd):
    """Borders of the dispatch at 152 multiprocessors: 1216 rows of 2048 columns, 608 of 4096, 9728 of 256, 19456 in eights."""
    forward(R, C, xd, rd, B, B)
    forward(R, C, xd, rd, F, F, pad=8)


@pytest.mark.parametrize("xd,rd", [(B, B), (F, None), (F, F)])
@pytest.mark.parametrize("R,C", [(1301, 2048), (701, 4096), (10001, 256), (1300, 5120), (333, 96)])
def test_rowwise_view_alone(R, C, xd, rd):
    x, w = matrix(R, C, xd), (1 + 0.2 * torch.randn(C, device=DEV)).to(B)
    x[R // 2] = 0
    x[R - 1, C - 1] = float("inf")
    kw = {} if rd is None else dict(residual=matrix(R, C, rd, 3.0), sum=torch.empty(R, C, dtype=rd, device=DEV))
    y, row = torch.empty(R, C, device=DEV), views(32 * (R // 32 + 1), C, False)[0]
    row = tuple(t[:R] for t in row)
    gtp.gtp_rmsnorm(x, w, 1e-5, y=y, row=row, **kw)
    check_view(row, y, False)
    again = tuple(torch.empty_like(t) for t in row)
    gtp.gtp_rmsnorm(x, w, 1e-5, row=again, **kw)
    assert all(torch.equal(a, b) for a, b in zip(row, again))


@pytest.mark.parametrize("xd,rd", [(B, B), (F, F)])
@pytest.mark.parametrize("R,C", [(1312, 4096), (2528, 2048)])
def test_views_of_many_rows(R, C, xd, rd):
    x, res, w = matrix(R, C, xd), matrix(R, C, rd, 3.0), (1 + 0.2 * torch.randn(C, device=DEV)).to(F)
    y, rstd, out = torch.empty(R, C, device=DEV), torch.empty(R, device=DEV), torch.empty(R, C, dtype=rd, device=DEV)
    row, col = views(R, C, True)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y, rstd=rstd, row=row, col=col)
    check_forward(out, w, 1e-5, rstd, y)
    check_view(row, y, True)
    check_view(col, y.t().contiguous(), True)


@pytest.mark.parametrize("dd,sd", [(B, B), (F, F), (B, F)])
@pytest.mark.parametrize("R,C", [(8191, 2048), (1001, 4096), (650, 8192), (611, 5120), (401, 16384), (3001, 12345), (1500, 5001), (1301, 2047),
                                 (5003, 31)])
def test_gradient_of_more_rows_than_blocks(R, C, dd, sd):
    gradient(R, C, dd, sd, F)


def sizes(R, C, dt):
    """Rows from 1e-18 to 3e38, each with a few elements far above its others, and some whose elements differ by decades; every
    fourth an ordinary one.  Scales are powers of two, so that bf16 holds them."""
    x = torch.randn(R, C, device=DEV).to(B).float()
    x[x == 0] = 1.0
    exponents = [60, 0, 63, 64, 65, 0, 90, 126, 100, 0, -58, 124]
    for r in range(R):
        x[r] *= 2.0 ** exponents[r % len(exponents)] / (8 if exponents[r % len(exponents)] > 120 else 1)
    for r in range(0, R, 5):  # one element holds the row's size
        x[r, (37 * r) % C] = -(2.0 ** 80)
    return x.to(dt)


def check_any(s, w, eps, rstd, y):
    from oracle import rmsnorm as N
    import numpy as np
    r, ref = N.forward(s.double().cpu().numpy(), w.double().cpu().numpy(), float(np.float32(eps)))
    got = rstd.double().cpu().numpy()
    tol = 26 * 2.0 ** -24 * r + 2.0 ** -149  # subnormal ones have a spacing of 2^-149
    assert np.all(np.abs(got - r) <= tol)
    assert np.all(r < 2.0 ** 128)
    tol = (29 * 2.0 ** -24 + 2.0 ** -149 / r[:, None]) * np.abs(ref)
    if y.dtype == B:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol + 2.0 ** -133)


# whole vectors and rows that start anywhere, by one warp and by many; from 1301 on several rows a thread, or more than a block
RANGES = [(1, 8), (40, 33), (13, 250), (30, 1000), (24, 2047), (14, 4001), (14, 8001), (13, 12345), (300, 72), (14, 4096),
          (13, 5120), (13, 16384), (1301, 2048), (701, 4096), (1301, 5120), (5003, 512), (13003, 100), (1500, 1001)]


@pytest.mark.parametrize("R,C", RANGES)
@pytest.mark.parametrize("xd,rd", [(B, None), (F, None), (B, B), (F, F)])
def test_rows_of_any_size(R, C, xd, rd):
    x, w = sizes(R, C, xd), (1 + 0.2 * torch.randn(C, device=DEV)).to(F)
    y, rstd = torch.full((R, C), float("nan"), device=DEV), torch.empty(R, device=DEV)
    kw, s = {}, x
    if rd is not None:
        res = x.to(rd) * 0.5
        s = torch.empty_like(res)
        kw = dict(residual=res, sum=s)
    for eps in (1e-5, 0.0, 1e-30):
        gtp.gtp_rmsnorm(x, w, eps, y=y, rstd=rstd, **kw)
        if rd is not None:
            assert torch.equal(s, (x.float() + res.float()).to(rd))
        check_any(s, w, eps, rstd, y)
    into = torch.full_like(y, float("nan")).to(xd) if rd is None else y
    gtp.gtp_rmsnorm(x, w, eps, y=into, **kw)
    # y in x's place, and the sum in the residual's
    want = [into.clone(), s.clone()]
    if rd is not None:
        kw["sum"] = s = kw["residual"]
    into = x if rd is None or rd == F else into
    gtp.gtp_rmsnorm(x, w, eps, y=into, **kw)
    assert torch.equal(into, want[0]) and (rd is None or torch.equal(s, want[1]))


@pytest.mark.parametrize("R,C", [(7, 8), (20, 250), (20, 256), (20, 1000), (20, 2048), (20, 4001), (14, 5120), (14, 9001)])
def test_small_rows_without_eps(R, C):
    """Squares below fp32's smallest number; eps so small that it is of the mean's size or the other way round."""
    w = 1 + 0.2 * torch.randn(C, device=DEV)
    x = torch.randn(R, C, device=DEV)
    for r in range(R):
        x[r] *= 2.0 ** (-50 - 11 * (r % 7))  # down to 2^-116
    y, rstd = torch.empty_like(x), torch.empty(R, device=DEV)
    for eps in (0.0, 2.0 ** -100, 2.0 ** -149, 2.0 ** -80):
        gtp.gtp_rmsnorm(x, w, eps, y=y, rstd=rstd)
        check_any(x, w, eps, rstd, y)


@pytest.mark.parametrize("xd,rd", [(B, B), (F, None), (B, None), (F, F)])
@pytest.mark.parametrize("R,C", [(32, 32), (64, 256), (64, 768), (64, 2016), (32, 2048), (64, 4096), (32, 8192)])
@pytest.mark.parametrize("tiled", [False, True])
def test_views_of_rows_of_any_size(R, C, xd, rd, tiled):
    x, w = sizes(R, C, xd), (1 + 0.2 * torch.randn(C, device=DEV)).to(B)
    kw, s = {}, x
    if rd is not None:
        res = x.to(rd) * 0.5
        s = torch.empty_like(res)
        kw = dict(residual=res, sum=s)
    for eps in (1e-5, 0.0):
        y, rstd = torch.empty(R, C, device=DEV), torch.empty(R, device=DEV)
        row, col = views(R, C, tiled)
        gtp.gtp_rmsnorm(x, w, eps, y=y, rstd=rstd, row=row, col=col, **kw)
        check_any(s, w, eps, rstd, y)
        check_view(row, y, tiled)
        check_view(col, y.t().contiguous(), tiled)
        # with the sum in x's or the residual's place
        if rd is not None:
            a, b, y2 = x.clone(), res.clone(), torch.empty_like(y)
            into = a if xd == rd else b
            gtp.gtp_rmsnorm(a, w, eps, residual=b, sum=into, y=y2, rstd=rstd, row=row, col=col)
            assert torch.equal(into, s) and torch.equal(y2, y)
