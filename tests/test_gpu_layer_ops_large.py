"""The embedding, the norm and the orthogonalised step on arrays of more than 2^31 elements or 2^32 bytes: offsets that pass
32 bits.  Sampled rows, the first and the last among them, at the tolerances of the operators' own tests."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import embedding as E
from oracle import mxfp8 as MX
from oracle import orthogonalize as O
from oracle import rmsnorm as N

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, F = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("C", [8192, 8191])
def test_embedding(C):
    """A table, an output and a gradient buffer of 2.3e9 elements each."""
    V = T = 280_000
    table = torch.empty(V, C, dtype=B, device=DEV).normal_()
    ids = torch.randint(0, V, (T,), device=DEV)
    ids[-3:] = V - 1
    ids[5] = V - 1
    out = torch.empty(T, C, dtype=B, device=DEV)
    gtp.gtp_embedding(ids, table, out, scale=0.5)
    for a in range(0, T, 40_000):  # a power of two: exact
        assert torch.equal(out[a:a + 40_000], table[ids[a:a + 40_000]] * 0.5)
    del table
    grad = torch.zeros(7 + V * C, device=DEV)
    ws = torch.empty(gtp.gtp_embedding_grad_workspace_bytes(T, V, C), dtype=torch.uint8, device=DEV)
    gtp.gtp_embedding_grad_accum(out, ids, grad, 7, V, ws, scale=0.5)
    host = ids.cpu().numpy()
    for r in (int(host[0]), int(host[T // 2]), V - 1):
        t = np.nonzero(host == r)[0]
        x = f64(out[torch.from_numpy(t).to(DEV)]) * 0.5
        err = np.abs(f64(grad[7 + r * C:7 + (r + 1) * C]) - x.sum(0))
        assert np.all(err <= (len(t) + 2) * U * np.abs(x).sum(0) + 1e-30)
    free_rows = np.setdiff1d(np.arange(V), host)[-3:]
    for r in free_rows:
        assert not grad[7 + int(r) * C:7 + (int(r) + 1) * C].any()
    assert not grad[:7].any()


@pytest.mark.parametrize("R,C", [(140_032, 16384), (280_000, 8191)])
def test_norm(R, C):
    x = torch.empty(R, C, dtype=B, device=DEV).normal_()
    w, rstd = 1 + 0.2 * torch.randn(C, device=DEV), torch.empty(R, device=DEV)
    y = torch.empty(R, C, dtype=B, device=DEV)
    row = col = None
    if C % 32 == 0:
        row, col = ((torch.empty(r, c, dtype=torch.uint8, device=DEV), torch.empty(r, c // 32, dtype=torch.uint8, device=DEV))
                    for r, c in ((R, C), (C, R)))
    gtp.gtp_rmsnorm(x, w, 1e-5, y=y, rstd=rstd, row=row, col=col)
    rows = [0, 1, R // 2, (1 << 31) // C, (1 << 31) // C + 1, R - 1]
    r, ref = N.forward(f64(x[rows]), f64(w), float(np.float32(1e-5)))
    assert np.all(np.abs(f64(rstd[rows]) - r) <= 26 * U * r)
    tol = 29 * U * np.abs(ref)
    assert np.all(np.abs(f64(y[rows]) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
    if row is not None:
        # a code's half step is 2^-4 of its value, 2^-3 where it saturates (512 to 448 of the scale); of the block's small
        # values half the smallest step, 2^-10 of the scale, which is at most the largest value over 256
        got, top = MX.dequantize_rowwise(*(t[rows].cpu().numpy() for t in row)), np.abs(ref).reshape(len(rows), -1, 32).max(2)
        assert np.all(np.abs(got - ref) <= (2.0 ** -3 + 1e-5) * np.abs(ref) + np.repeat(top, 32, 1) * 2.0 ** -17)
        cols, part = [0, C // 2, C - 1], slice(R - 64, R)
        _, ref = N.forward(f64(x[part]), f64(w), float(np.float32(1e-5)))
        ref = ref.T[cols]
        got = MX.dequantize_rowwise(*(t[cols][:, -n:].cpu().numpy() for t, n in zip(col, (64, 2))))
        top = np.abs(ref).reshape(len(cols), -1, 32).max(2)
        assert np.all(np.abs(got - ref) <= (2.0 ** -3 + 1e-5) * np.abs(ref) + np.repeat(top, 32, 1) * 2.0 ** -17)
        back = torch.empty(R, C, dtype=B, device=DEV)
        gtp.gtp_mxfp8_dequantize(*row, back)
        assert np.array_equal(f64(back[rows]), MX.dequantize_rowwise(*(t[rows].cpu().numpy() for t in row)))
        del back, row, col
    dx, grad = torch.empty_like(y), torch.zeros(C, device=DEV)
    ws = torch.empty(gtp.gtp_rmsnorm_grad_workspace_bytes(R, C), dtype=torch.uint8, device=DEV)
    gtp.gtp_rmsnorm_grad(y, x, rstd, w, dx, grad, 0, ws)
    rdx, _ = N.gradient(f64(y[rows]), f64(x[rows]), f64(rstd[rows]), f64(w))
    rr = f64(rstd[rows])[:, None]
    n, g = np.abs(f64(x[rows]) * rr), np.abs(f64(y[rows]) * f64(w))
    tol = rr * (4 * U * g + n * (n * g).mean(1, keepdims=True) * 52 * U) + 2 * U * np.abs(rdx)
    assert np.all(np.abs(f64(dx[rows]) - rdx) <= tol + 2.0 ** -8 * (np.abs(rdx) + tol))
    # all rows' sum: torch's, in fp64 by parts
    want, mass = torch.zeros(C, dtype=torch.float64, device=DEV), torch.zeros(C, dtype=torch.float64, device=DEV)
    for a in range(0, R, 20_000):
        t = y[a:a + 20_000].double() * x[a:a + 20_000].double() * rstd[a:a + 20_000, None].double()
        want += t.sum(0)
        mass += t.abs().sum(0)
    assert ((grad.double() - want).abs() <= (R + 40) * U * mass).all()


def test_step_behind_32_bits():
    R, C = 130, 257
    at = (1 << 31) + 12345
    n = at + R * C + 3
    grad, m, p = (torch.zeros(n, device=DEV) for _ in range(3))
    param = torch.zeros(n, dtype=B, device=DEV)
    offsets = [at, 5]
    for k, o in enumerate(offsets):
        grad[o:o + R * C] = 1e-3 * torch.randn(R * C, device=DEV)
        p[o:o + R * C] = 0.02 * torch.randn(R * C, device=DEV)
    g0, p0 = ([f64(t[o:o + R * C]).reshape(R, C) for o in offsets] for t in (grad, p))
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(2, R, C), dtype=torch.uint8, device=DEV)
    gtp.gtp_muon_step(grad, m, p, param, offsets, R, C, gtp.MuonHparams(lr=0.02, momentum=0.9, weight_decay=0.1, scale=1.5), ws)
    for o, g, q in zip(offsets, g0, p0):
        _, w = O.step(g, np.zeros((R, C)), q, float(np.float32(0.9)), 0.02, 0.1, 1.5)
        got = p[o:o + R * C]
        assert np.linalg.norm(f64(got).reshape(R, C) - w) <= 4e-3 * np.linalg.norm(w - q * (1 - 0.002)) + 2.0 ** -22 * np.linalg.norm(q)
        assert torch.equal(param[o:o + R * C], got.to(B)) and not grad[o:o + R * C].any()
        p[o:o + R * C] = 0
    assert not p.any()  # nothing beside the views


def test_orthogonalize_rows_far_apart():
    """A matrix whose rows and planes lie 2^32 bytes and more apart."""
    R, C, ld = 70, 40, 1 << 26
    src = torch.empty(2, R, ld, dtype=B, device=DEV)[:, :, ld - C:]
    src.normal_()
    out = torch.empty(2, R, C, device=DEV)
    gtp.gtp_orthogonalize(src, out, torch.empty(gtp.gtp_orthogonalize_workspace_bytes(2, R, C), dtype=torch.uint8, device=DEV))
    for k in range(2):
        want = O.orthogonalize(f64(src[k]))
        assert np.linalg.norm(f64(out[k]) - want) <= 4e-3 * np.linalg.norm(want)


@pytest.mark.parametrize("R,C", [(65536, 16), (16, 65536), (3, 65536), (65536, 200), (300, 30000), (30000, 260)])
def test_orthogonalize_long_sides(R, C):
    src = 1e-3 * torch.randn(R, C, device=DEV)
    out = torch.full((R, C), float("nan"), device=DEV)
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(1, R, C), dtype=torch.uint8, device=DEV).fill_(0xFF)
    gtp.gtp_orthogonalize(src, out, ws)
    want = O.orthogonalize(f64(src))
    assert np.linalg.norm(f64(out) - want) <= 4e-3 * np.linalg.norm(want)
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("R,C", [(257, 270), (130, 40)])
def test_a_step_of_64_weights(R, C):
    n, each = 64, R * C
    offsets = [k * (each + 1) for k in range(n)]
    g, m, p = (torch.randn(n * (each + 1), device=DEV) * s for s in (1e-3, 1e-3, 0.02))
    g0, m0, p0 = g.clone(), m.clone(), p.clone()
    ws = torch.empty(gtp.gtp_orthogonalize_workspace_bytes(n, R, C), dtype=torch.uint8, device=DEV).fill_(0xFF)
    h = gtp.MuonHparams(lr=0.02, momentum=0.9, weight_decay=0.1, scale=1.5)
    gtp.gtp_muon_step(g, m, p, None, offsets, R, C, h, ws)
    for k in (0, 1, 31, 62, 63):
        view = lambda t: f64(t[offsets[k]:offsets[k] + each]).reshape(R, C)
        _, w = O.step(view(g0), view(m0), view(p0), float(np.float32(0.9)), 0.02, 0.1, 1.5)
        moved = np.linalg.norm(w - view(p0) * (1 - 0.002))
        assert np.linalg.norm(view(p) - w) <= 4e-3 * moved + 2.0 ** -22 * np.linalg.norm(view(p0))
    gap = torch.tensor([o + each for o in offsets], device=DEV)
    assert torch.equal(p[gap], p0[gap]) and torch.equal(m[gap], m0[gap]) and torch.equal(g[gap], g0[gap])
    assert gtp.gtp_wait_timeouts() == 0
