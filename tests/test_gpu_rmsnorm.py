"""The norm, its views and its gradient on the GPU against the float64 oracle.

The sum is one fp32 addition rounded once: compared bit for bit.  rstd: a row's sum of squares is formed by at most 32
multiply-adds a thread and 12 additions across, 44 roundings of positive terms whose effect the root halves, then a
division, an addition, a root and a reciprocal: 26 * 2^-24 relative.  y: rstd's error and two products, half a bf16 step
(2^-8) where bf16.  The views are those of the fp32 y, bit for bit.  dx = rstd (g - n mean) + dsum: g, n and the products
2^-24 each, the mean as above over |g n|.  The weight's gradient: one rounding a row and the additions across."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import mxfp8 as MX
from oracle import rmsnorm as N
from oracle import sf_layout as SF

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def matrix(R, C, dt, scale=1.0, pad=0, shift=0):
    """A [R, C] view, its rows pad elements further apart than they are long and shift elements in."""
    return (torch.randn(R, C + pad + shift, device=DEV) * scale).to(dt)[:, shift:shift + C]


def check_forward(s, w, eps, rstd, y):
    r, ref = N.forward(f64(s), f64(w), float(np.float32(eps)))
    assert np.all(np.abs(f64(rstd) - r) <= 26 * U * r)
    tol = 29 * U * np.abs(ref)
    if y.dtype == B:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert np.all(np.abs(f64(y) - ref) <= tol + 2.0 ** -133)


def forward(R, C, xd, rd, wd, yd, pad=0, shift=0):
    x, w = matrix(R, C, xd, pad=pad, shift=shift), (1 + 0.2 * torch.randn(C, device=DEV)).to(wd)
    y, rstd = torch.full((R, C), float("nan"), dtype=yd, device=DEV), torch.empty(R, device=DEV)
    if rd is None:
        gtp.gtp_rmsnorm(x, w, 1e-5, y=y, rstd=rstd)
        check_forward(x, w, 1e-5, rstd, y)
        return
    res = matrix(R, C, rd, 3.0, 2 * pad, shift)
    out = torch.full((R, C + pad), float("nan"), dtype=rd, device=DEV)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out[:, :C], y=y, rstd=rstd)
    assert torch.equal(out[:, :C], (x.float() + res.float()).to(rd))
    assert torch.isnan(out[:, C:].float()).all()
    check_forward(out[:, :C], w, 1e-5, rstd, y)


@pytest.mark.parametrize("xd,rd", [(B, None), (F, None), (B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 33), (1, 2048), (700, 2048), (1500, 256), (9, 1535), (2, 16384),
                                 (5, 4104), (650, 520), (4, 12345)])
def test_forward(R, C, xd, rd):
    for wd, yd in ((B, B), (F, F)):
        forward(R, C, xd, rd, wd, yd)


@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 0), (0, 3), (16, 8), (1, 1)])
def test_strides_and_alignment(pad, shift):
    for xd, rd in ((B, B), (F, B), (B, F), (F, None)):
        forward(33, 72, xd, rd, B, B, pad, shift)


def test_in_place_and_rows_of_zeros_and_nan():
    x, res, w = torch.randn(40, 96, device=DEV), torch.randn(40, 96, device=DEV), torch.ones(96, device=DEV)
    x[3], res[3] = 0, 0
    x[7, 5], res[9, 95] = float("nan"), float("inf")
    want, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(40, device=DEV)
    gtp.gtp_rmsnorm(x, w, 1e-6, residual=res, sum=want, y=y, rstd=rstd)
    assert not y[3].any() and rstd[3].item() == pytest.approx(1000.0, rel=1e-6)
    assert torch.isnan(y[7]).all() and torch.isnan(rstd[7]) and torch.isnan(y[9, 95]) and not y[9, :95].any()
    others = [i for i in range(40) if i not in (7, 9)]
    assert torch.isfinite(y[others]).all()
    gtp.gtp_rmsnorm(torch.zeros(2, 8, device=DEV), torch.ones(8, device=DEV), 0.0, y=(z := torch.empty(2, 8, device=DEV)))
    assert torch.isnan(z).all()  # 0 * Inf, as the formula says with eps 0
    for into in ("residual", "x"):
        a, b, got = x.clone(), res.clone(), torch.empty_like(x)
        gtp.gtp_rmsnorm(a, w, 1e-6, residual=b, sum=b if into == "residual" else a, y=got)
        assert torch.equal((b if into == "residual" else a)[others], want[others])
        assert torch.equal(got[others], y[others])
    a = x.clone()
    gtp.gtp_rmsnorm(a, w, 1e-6, y=a)
    b = torch.empty_like(x)
    gtp.gtp_rmsnorm(x, w, 1e-6, y=b)
    assert torch.equal(a[others], b[others])


def views(R, C, tiled):
    u8 = dict(dtype=torch.uint8, device=DEV)

    def one(r, c):
        n = gtp.gtp_sf_tiled_bytes(r, c // 32)
        return torch.empty(r, c, **u8), torch.zeros(n, **u8) if tiled else torch.empty(r, c // 32, **u8)
    return one(R, C), one(C, R)


def check_view(view, y, tiled):
    codes, scales = MX.quantize_rowwise(y.cpu().numpy())
    assert np.array_equal(view[0].cpu().numpy(), codes)
    want = SF.tile_scales(scales).ravel() if tiled else scales
    assert np.array_equal(view[1].cpu().numpy(), want)


@pytest.mark.parametrize("xd,rd", [(B, B), (F, None), (B, F), (F, B), (B, None), (F, F)])
@pytest.mark.parametrize("R,C", [(32, 32), (64, 256), (96, 288), (64, 2048), (32, 2080), (64, 4096), (32, 4128), (32, 16384)])
@pytest.mark.parametrize("tiled", [False, True])
def test_views(R, C, xd, rd, tiled):
    x, w = matrix(R, C, xd), (1 + 0.2 * torch.randn(C, device=DEV)).to(B)
    x[:, 5] *= 100
    x[1, 32 * (C // 64)] = float("nan") if R > 64 else 1.0
    x[2] = 0
    res = None if rd is None else matrix(R, C, rd, 3.0)
    if rd is not None:
        res[2] = 0
    out = None if rd is None else torch.empty(R, C, dtype=rd, device=DEV)
    y, rstd = torch.empty(R, C, device=DEV), torch.empty(R, device=DEV)
    row, col = views(R, C, tiled)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y, rstd=rstd, row=row, col=col)
    s = x if rd is None else out
    if R <= 64:
        check_forward(s, w, 1e-5, rstd, y)
    check_view(row, y, tiled)
    check_view(col, y.t().contiguous(), tiled)
    # Each view by itself, of the y of its own call: which outputs are asked for decides the order in which a row's squares
    # are summed, so two calls' rstd may differ within its error above and with it a code next to a border.
    row2, col2 = views(R, C, tiled)
    y2 = torch.empty(R, C, device=DEV)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y2, row=row2)
    check_view(row2, y2, tiled)
    row3, _ = views(R, C, tiled)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, row=row3)
    gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, rstd=rstd, col=col2)
    for a, b in ((row2, row3), (col, col2)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # the views' values
    for view, of in ((row, y), (col, y.t())):
        got32, got16 = torch.empty(of.shape, device=DEV), torch.empty(of.shape, dtype=B, device=DEV)
        gtp.gtp_mxfp8_dequantize(*view, got32)
        gtp.gtp_mxfp8_dequantize(*view, got16)
        want = MX.dequantize_rowwise(*MX.quantize_rowwise(of.contiguous().cpu().numpy()))
        assert np.array_equal(f64(got32), want, equal_nan=True) and np.array_equal(f64(got16), want, equal_nan=True)


@pytest.mark.parametrize("dd,sd", [(B, B), (B, F), (F, F), (F, B)])
@pytest.mark.parametrize("R,C", [(1, 1), (1, 8), (3, 33), (700, 2048), (1500, 256), (9, 1535), (2, 16384), (5, 4104), (4, 12345),
                                 (3000, 72)])
@pytest.mark.parametrize("gd", [F, B])
def test_gradient(R, C, dd, sd, gd):
    for with_dsum, pad, shift in ((True, 0, 0), (False, 0, 0), (True, 8, 0), (True, 3, 1)):
        dy, s = matrix(R, C, dd, 1.0, pad, shift), matrix(R, C, sd, 2.0, 2 * pad, shift)
        ds = matrix(R, C, sd, 1.0, pad, shift) if with_dsum else None
        w = (1 + 0.2 * torch.randn(C, device=DEV)).to(F if pad else B)
        rstd = torch.rsqrt(s.float().square().mean(1) + 1e-5)
        dx = torch.full((R, C + pad), float("nan"), dtype=sd, device=DEV)
        grad = torch.randn(C + 8, device=DEV).to(gd)
        before = grad.clone()
        ws = torch.empty(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
        ws.fill_(0x7F)
        gtp.gtp_rmsnorm_grad(dy, s, rstd, w, dx[:, :C], grad, 5, ws, dsum=ds)
        rdx, rdw = N.gradient(f64(dy), f64(s), f64(rstd), f64(w), None if ds is None else f64(ds))
        r = f64(rstd)[:, None]
        n, g = np.abs(f64(s) * r), np.abs(f64(dy) * f64(w))
        mean = (n * g).mean(1, keepdims=True)
        tol = r * (4 * U * g + n * mean * 52 * U) + 2 * U * (np.abs(rdx) + (0 if ds is None else np.abs(f64(ds))))
        if sd == B:
            tol = tol + 2.0 ** -8 * (np.abs(rdx) + tol)
        assert np.all(np.abs(f64(dx[:, :C]) - rdx) <= tol + 2.0 ** -133)
        assert torch.isnan(dx[:, C:].float()).all()
        ref = f64(before[5:5 + C]) + rdw
        mass = (np.abs(f64(dy)) * n).sum(0)
        tol = (R + 40) * U * mass + U * np.abs(ref)
        if gd == B:
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
        assert np.all(np.abs(f64(grad[5:5 + C]) - ref) <= tol)
        assert torch.equal(grad[:5], before[:5]) and torch.equal(grad[5 + C:], before[5 + C:])


def test_gradient_is_the_forward_s_difference():
    R, C, h = 6, 40, 1e-3
    x, w, dy = torch.randn(R, C, device=DEV), 1 + 0.2 * torch.randn(C, device=DEV), torch.randn(R, C, device=DEV)
    along, along_w = torch.randn(R, C, device=DEV), torch.randn(C, device=DEV)

    def loss(t):
        y = torch.empty(R, C, device=DEV)
        gtp.gtp_rmsnorm(x + t * along, w + t * along_w, 1e-5, y=y)
        return (y.double() * dy.double()).sum().item()
    rstd, y, dx, grad = torch.empty(R, device=DEV), torch.empty(R, C, device=DEV), torch.empty(R, C, device=DEV), torch.zeros(C, device=DEV)
    gtp.gtp_rmsnorm(x, w, 1e-5, y=y, rstd=rstd)
    ws = torch.empty(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
    gtp.gtp_rmsnorm_grad(dy, x, rstd, w, dx, grad, 0, ws)
    slope = ((dx.double() * along.double()).sum() + (grad.double() * along_w.double()).sum()).item()
    # the values' rounding over the step (2 h apart) and the third derivative's h^2, both about 1e-3 of R C terms
    assert abs((loss(h) - loss(-h)) / (2 * h) - slope) <= 2e-3 * R * C


def test_gradient_in_place_and_equal_bits():
    R, C = 300, 1024
    dy, s, ds = (torch.randn(R, C, device=DEV).to(B) for _ in range(3))
    w, rstd = torch.randn(C, device=DEV), torch.rand(R, device=DEV)
    ws = torch.empty(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
    dx, grad = torch.empty_like(s), torch.zeros(C, device=DEV)
    gtp.gtp_rmsnorm_grad(dy, s, rstd, w, dx, grad, 0, ws, dsum=ds)
    for k in range(3):
        ops = [dy.clone(), s.clone(), ds.clone()]
        again = torch.zeros(C, device=DEV)
        gtp.gtp_rmsnorm_grad(ops[0], ops[1], rstd, w, ops[k], again, 0, ws, dsum=ops[2])
        assert torch.equal(ops[k], dx) and torch.equal(again, grad)


def test_captured_on_a_side_stream():
    R, C = 64, 512
    x, res, w, dy = (torch.randn(*s, device=DEV) for s in ((R, C), (R, C), (C,), (R, C)))
    out, y, rstd, dx, grad = torch.empty(R, C, device=DEV), torch.empty(R, C, device=DEV), torch.empty(R, device=DEV), \
        torch.empty(R, C, device=DEV), torch.zeros(C, device=DEV)
    row, col = views(R, C, True)
    ws = torch.empty(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)

    def go():
        gtp.gtp_rmsnorm(x, w, 1e-5, residual=res, sum=out, y=y, rstd=rstd, row=row, col=col)
        gtp.gtp_rmsnorm_grad(dy, out, rstd, w, dx, grad, 0, ws, dsum=y)
    go()
    want = [t.clone() for t in (out, y, rstd, dx, grad, *row, *col)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        go()
    for t in (out, y, rstd, dx, grad):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (out, y, rstd, dx, grad, *row, *col)))
