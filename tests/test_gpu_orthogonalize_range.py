"""The orthogonalised update and its step on elements of any finite size, on the GPU against float64: squares that leave
fp32's range, norms whose reciprocal does.  Tolerances as test_gpu_orthogonalize_accuracy.py derives them."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import orthogonalize as O
from test_gpu_orthogonalize import B, DEV, F, f64, rel, workspace

pytestmark = pytest.mark.gpu
TOL = 1.5e-3  # five steps, Gaussian matrices


def gauss(R, C, seed):
    return torch.randn(R, C, generator=torch.Generator().manual_seed(seed + R + C))


def run(src):
    out = torch.full(src.shape, float("nan"), device=DEV)
    gtp.gtp_orthogonalize(src, out, workspace(1, *src.shape))
    assert rel(out, O.orthogonalize(f64(src))) <= TOL


@pytest.mark.parametrize("R,C", [(40, 72), (33, 17), (300, 520), (200, 1000)])
@pytest.mark.parametrize("exponent", [-149, -140, -127, -110, -90, -76, -74, -72, -63, -50, 50, 59, 61, 63, 64, 90, 124])
def test_one_size(R, C, exponent):
    x = gauss(R, C, 1).double() * 2.0 ** exponent
    if exponent < -126:
        x = x * 16  # subnormal numbers of a few bits and more
    run(x.float().to(DEV))
    if -120 < exponent:
        run(x.float().to(B).to(DEV))


@pytest.mark.parametrize("R,C", [(64, 128), (257, 301)])
def test_many_sizes(R, C):
    """Parts whose squares fp32 holds beside parts whose squares it does not; zeros."""
    x = gauss(R, C, 2)
    big = x.clone()
    big[:R // 2] *= 2.0 ** 63
    run(big.to(DEV))
    small = x * 2.0 ** -80
    small[R // 3] *= 2.0 ** 8
    small[:, ::3] = 0
    run(small.to(DEV))
    one = torch.zeros(R, C)
    one[R - 1, 3] = -(2.0 ** -140)
    run(one.to(DEV))
    out = torch.full((R, C), float("nan"), device=DEV)
    gtp.gtp_orthogonalize(torch.zeros(R, C, device=DEV), out, workspace(1, R, C))
    assert not out.any()


@pytest.mark.parametrize("exponent", [-120, -74, 60, 100])
def test_step(exponent):
    R, C = 96, 160
    grad, m, p = ((gauss(R, C, k) * 2.0 ** exponent).flatten().to(DEV) for k in range(3))
    p = p * 2.0 ** -exponent
    g0, m0, p0 = (f64(t).reshape(R, C) for t in (grad, m, p))
    h = gtp.MuonHparams(lr=0.5, momentum=0.9, weight_decay=0.0, scale=1.0)
    gtp.gtp_muon_step(grad, m, p, None, [0], R, C, h, workspace(1, R, C))
    wm, wp = O.step(g0, m0, p0, float(np.float32(0.9)), 0.5, 0.0, 1.0)
    assert np.all(np.abs(f64(m).reshape(R, C) - wm) <= 2.0 ** -22 * (np.abs(m0) + np.abs(g0)) + 2.0 ** -148)
    assert np.linalg.norm(f64(p).reshape(R, C) - wp) <= TOL * np.linalg.norm(wp - p0) + 2.0 ** -23 * np.linalg.norm(p0)
    assert not grad.any()
