"""The orthogonalised update and the step on it on the GPU against the float64 oracle.

What is rounded, at half a step of fp16 (2^-11) unless said: the products' X, the off-diagonal parts of A and of
b A + c A^2, each iteration; the linear term's X to 2^-22.  One iteration alone: the X that the product reads is off by
2^-11 / sqrt(3) of itself at most in the mean square, B by as much and by A's own error times |b| + 2 c < 9, all under
|B| + |E| of a few: 4e-3 of the result.  Five iterations of those errors, each carried on by slopes between 3.4 (small
singular values, which grow as much themselves) and -1.1 (those near 1): simulated with every rounding on Gaussian,
row-scaled and low-rank matrices 3e-4 to 1.5e-3, so 4e-3 here as well.  A bf16 result adds 2^-8 at most."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import orthogonalize as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32
TOL = 4e-3


def f64(t):
    return t.double().cpu().numpy()


def workspace(count, R, C, extra=0):
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(count, R, C) + extra, dtype=torch.uint8, device=DEV)
    return ws.fill_(0xFF)  # NaN wherever something would be read before it is written


def gradient(*shape, kind="gauss", seed=0):
    g = torch.Generator().manual_seed(seed + sum(shape))
    x = torch.randn(*shape, generator=g)
    if kind == "low rank":
        k = min(8, *shape)
        x = torch.randn(shape[0], k, generator=g) @ torch.randn(k, shape[1], generator=g) + 0.1 * x
    if kind == "rows":
        x = x * torch.exp(torch.randn(shape[0], 1, generator=g))
    return (1e-3 * x).to(DEV)


def rel(got, want):
    return np.linalg.norm(f64(got) - want) / max(np.linalg.norm(want), 1e-300)


def check(got, src, **how):
    want = O.orthogonalize(f64(src), **how)
    tol = TOL + (2.0 ** -8 if got.dtype == B else 0)
    assert rel(got, want) <= tol
    # no element or tile of its own: the worst is of the size that rounding noise has
    rms = np.sqrt(np.mean(want ** 2))
    assert np.abs(f64(got) - want).max() <= 12 * tol * max(rms, np.abs(want).max())


@pytest.mark.parametrize("R,C", [(1, 1), (1, 40), (40, 1), (16, 16), (17, 33), (33, 17), (64, 64), (130, 257), (257, 130), (512, 256),
                                 (300, 1000), (777, 1111), (1111, 777), (256, 2048), (2048, 264)])
@pytest.mark.parametrize("steps", [1, 5])
def test_shapes(R, C, steps):
    for kind, sd, od in (("gauss", F, F), ("low rank", B, B), ("rows", F, B)):
        src = gradient(R, C, kind=kind).to(sd)
        out = torch.full((R, C), float("nan"), dtype=od, device=DEV)
        gtp.gtp_orthogonalize(src, out, workspace(1, R, C), steps=steps)
        check(out, src, steps=steps)
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("count,R,C", [(1, 256, 300), (1, 200, 129), (2, 129, 200), (1, 70, 300), (3, 300, 70), (1, 60, 500), (1, 500, 60),
                                       (1, 128, 1000), (2, 1000, 128), (1, 65, 129), (1, 193, 2000), (1, 2000, 193), (1, 256, 256),
                                       (20, 256, 300), (20, 300, 200), (70 // 2, 128, 300)])
def test_small_sides(count, R, C):
    """Where a Gram matrix is one tile: X's tiles whole and in halves, alone and shared."""
    src = torch.stack([gradient(R, C, seed=k) for k in range(count)])
    out = torch.full_like(src, float("nan"))
    gtp.gtp_orthogonalize(src, out, workspace(count, R, C))
    for k in range(count):
        check(out[k], src[k])
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("count,R,C", [(3, 100, 200), (5, 200, 100), (2, 513, 512), (64, 8, 24), (3, 700, 600), (7, 300, 520), (9, 264, 264),
                                       (2, 1500, 1040)])
def test_stacks(count, R, C):
    src = torch.stack([gradient(R, C, seed=k) * 10.0 ** k if k < 8 else gradient(R, C, seed=k) for k in range(count)])
    src[1] = 0
    out = torch.full_like(src, float("nan"))
    gtp.gtp_orthogonalize(src, out, workspace(count, R, C))
    for k in range(count):
        check(out[k], src[k])
    assert not out[1].any()
    again = src.clone()
    gtp.gtp_orthogonalize(again, again, workspace(count, R, C))  # in place, and the same bits
    assert torch.equal(again, out)


def test_strides_and_borders():
    src = torch.zeros(3, 70, 150, device=DEV)
    src[:, 1:66, 3:104] = torch.stack([gradient(65, 101, seed=k) for k in range(3)])
    out = torch.full((3, 80, 120), 9.0, device=DEV).to(B)
    gtp.gtp_orthogonalize(src[:, 1:66, 3:104], out[:, 2:67, 5:106], workspace(3, 65, 101))
    for k in range(3):
        check(out[k, 2:67, 5:106], src[k, 1:66, 3:104])
    edge = out.clone()
    edge[:, 2:67, 5:106] = 9
    assert torch.all(edge == 9)


def test_values_that_are_not_finite_and_extreme_sizes():
    for bad in (float("nan"), float("inf")):
        src = torch.stack([gradient(40, 70), gradient(40, 70)])
        src[0, 3, 5] = bad
        out = torch.zeros_like(src)
        gtp.gtp_orthogonalize(src, out, workspace(2, 40, 70))
        assert torch.isnan(out[0]).all()
        check(out[1], src[1])  # its neighbour in the stack is its own
    for size in (1e-15, 1e15):
        src = gradient(40, 70) * size
        out = torch.empty_like(src)
        gtp.gtp_orthogonalize(src, out, workspace(1, 40, 70))
        check(out, src)
    one = torch.zeros(50, 60, device=DEV)
    one[7, 9] = -4.0  # a single element holds the whole norm
    out = torch.empty_like(one)
    gtp.gtp_orthogonalize(one, out, workspace(1, 50, 60))
    check(out, one)


def test_other_coefficients():
    src = gradient(90, 200)
    out = torch.empty_like(src)
    gtp.gtp_orthogonalize(src, out, workspace(1, 90, 200), steps=12, coefficients=(1.5, -0.5, 0.0))
    check(out, src, steps=12, coefficients=(1.5, -0.5, 0.0))


@pytest.mark.parametrize("gd,nesterov", [(F, True), (B, True), (F, False)])
@pytest.mark.parametrize("count,R,C,odd", [(1, 96, 160, 0), (3, 160, 96, 0), (2, 77, 111, 1), (4, 64, 64, 8)])
def test_step(count, R, C, odd, gd, nesterov):
    each = R * C
    offsets = [odd + k * (each + 64 + odd) for k in range(count)][::-1]
    n = count * (each + 64 + odd) + odd + 5
    g = torch.Generator(device=DEV).manual_seed(n)
    grad, m, p = (torch.randn(n, generator=g, device=DEV) * s for s in (1e-3, 1e-3, 0.02))
    grad = grad.to(gd)
    param = torch.full((n,), 3.0, device=DEV).to(B)
    before = [t.clone() for t in (grad, m, p, param)]
    clip = torch.tensor([0.5], device=DEV)
    h = gtp.MuonHparams(lr=0.02, momentum=0.9, weight_decay=0.1, scale=1.5, grad_factor=0.25, nesterov=nesterov)
    gtp.gtp_muon_step(grad, m, p, param, offsets, R, C, h, workspace(count, R, C), grad_scale=clip)
    inside = torch.zeros(n, dtype=torch.bool, device=DEV)
    for at in offsets:
        inside[at:at + each] = True
        g0, m0, p0 = (f64(t[at:at + each]).reshape(R, C) for t in before[:3])
        wm, _ = O.step(g0 * 0.125, m0, p0, float(np.float32(0.9)), 0.0, 0.0, 0.0, nesterov)
        gm = f64(m[at:at + each]).reshape(R, C)
        assert np.all(np.abs(gm - wm) <= 2.0 ** -22 * (np.abs(m0) + np.abs(g0)))
        wm, wp = O.step(g0 * 0.125, m0, p0, float(np.float32(0.9)), float(np.float32(0.02)), float(np.float32(0.1)), 1.5, nesterov)
        got, moved = f64(p[at:at + each]).reshape(R, C), wp - p0 * (1 - 0.02 * 0.1)
        assert np.linalg.norm(got - wp) <= TOL * np.linalg.norm(moved) + 2.0 ** -22 * np.linalg.norm(p0)
        assert torch.equal(param[at:at + each], p[at:at + each].to(B))
        assert not grad[at:at + each].any()
    for t, b in zip((grad, m, p, param), before):  # nothing beside the views
        assert torch.equal(t[~inside], b[~inside])


def test_step_keeps_gradients_and_goes_without_param():
    R, C = 48, 80
    grad, m, p = torch.randn(R * C, device=DEV), torch.zeros(R * C, device=DEV), torch.randn(R * C, device=DEV)
    before = grad.clone()
    gtp.gtp_muon_step(grad, m, p, None, [0], R, C, gtp.MuonHparams(zero_grad_after=False), workspace(1, R, C))
    assert torch.equal(grad, before)
    q, m2 = p.clone(), m.clone()
    param = torch.empty(R * C, dtype=B, device=DEV)
    gtp.gtp_muon_step(grad, m, p, param, [0], R, C, gtp.MuonHparams(lr=0.0, zero_grad_after=False), workspace(1, R, C))
    assert torch.equal(p, q) and torch.equal(param, p.to(B)) and not torch.equal(m, m2)


def test_captured_on_a_side_stream():
    R, C = 200, 300
    src, out = gradient(R, C), torch.empty(R, C, device=DEV)
    ws = workspace(1, R, C)
    gtp.gtp_orthogonalize(src, out, ws)
    want = out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        gtp.gtp_orthogonalize(src, out, ws)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert gtp.gtp_wait_timeouts() == 0
