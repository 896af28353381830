"""The orthogonalised update's accuracy on the GPU against float64, as the header states it.

The bounds come from the kernels' roundings restated in float64 (fp16 X, A' and B', X's low part scaled by a in all but the
last three iterations), worst over the families below on sides of 40 to 2000: 9.9e-4 at five steps (2.6e-3 on rank 8 with 1e-3
of noise, 1.3e-3 on spread singular values), 2.5e-3 at six, 2e-3 at eight, 3e-3 at ten, 5.5e-3 at twelve, 1.2e-2 at sixteen;
half as much again for other draws.  The error is spread evenly: a block of 32 x 32 has at most 1.8 times the mean square's
root, so four times the bound holds for each block, the narrow ones at the edges among them."""
import numpy as np
import pytest
import torch

import param_buffers_gb300 as gtp
from oracle import orthogonalize as O
from test_gpu_orthogonalize import DEV, F, f64, workspace

pytestmark = pytest.mark.gpu
BOUND = {1: 5e-4, 5: 1.5e-3, 6: 4e-3, 8: 4e-3, 10: 4.5e-3, 12: 8e-3, 16: 2e-2}


def matrix(m, n, kind, seed):
    g = torch.Generator().manual_seed(seed + 7 * m + n)
    randn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    x = randn(m, n)
    if kind == "rows":
        x = x * torch.exp(randn(m, 1))
    elif kind.startswith("noise"):  # rank 8 and so much of everything else
        x = randn(m, 8) @ randn(8, n) + float(kind.split()[1]) * x
    elif kind.startswith("spread"):  # singular values from 1 down, evenly in their logarithm
        k = min(m, n)
        u, v = torch.linalg.qr(randn(m, k))[0], torch.linalg.qr(randn(n, k))[0]
        x = (u * torch.logspace(0, float(kind.split()[1]), k, dtype=torch.float64)) @ v.T
    return (1e-3 * x).float().to(DEV)


def check(m, n, kind, steps, bound, seed=0):
    src = matrix(m, n, kind, seed)
    out = torch.full((m, n), float("nan"), dtype=F, device=DEV)
    gtp.gtp_orthogonalize(src, out, workspace(1, m, n), steps=steps)
    want = O.orthogonalize(f64(src), steps=steps)
    off = f64(out) - want
    assert np.linalg.norm(off) <= bound * np.linalg.norm(want), (kind, np.linalg.norm(off) / np.linalg.norm(want))
    rms = np.sqrt(np.mean(want ** 2))
    worst = max(np.sqrt(np.mean(off[i:i + 32, j:j + 32] ** 2)) for i in range(0, m, 32) for j in range(0, n, 32))
    assert worst <= 4 * bound * rms, (kind, worst / rms)


SHAPES = [(40, 70), (96, 1024), (1024, 96), (256, 300), (512, 512), (700, 777), (777, 700), (300, 2000), (2000, 300)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("steps", [1, 5])
def test_usual_matrices(m, n, steps):
    for kind in ("gauss", "rows", "noise 0.1", "spread -2"):
        check(m, n, kind, steps, BOUND[steps])
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("m,n", SHAPES)
def test_a_few_directions_that_hold_nearly_all(m, n):
    for kind in ("noise 0.001", "spread -4", "spread -6"):
        check(m, n, kind, 5, 3e-3)
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("steps", [6, 8, 10, 12, 16])
def test_more_steps(m, n, steps):
    for kind in ("gauss", "noise 0.1", "noise 0.001", "spread -2", "spread -4", "spread -6"):
        check(m, n, kind, steps, BOUND[steps])
    assert gtp.gtp_wait_timeouts() == 0


@pytest.mark.parametrize("m,n,bound", [(1, 1, 1e-3), (1, 40, 4e-3), (2, 2, 1.5e-2), (3, 2, 1.5e-2), (2, 100, 1.5e-2), (20, 3, 1.5e-2), (4, 4, 1.5e-2),
                                       (8, 8, 6e-3), (64, 8, 6e-3), (16, 16, 2.5e-3), (16, 64, 2.5e-3), (100, 32, 2e-3), (64, 64, 1.6e-3)])
def test_short_sides(m, n, bound):
    """Few elements do not average their roundings out: of 400 simulated draws at five steps the worst 9e-3 with a side of 2,
    3.2e-3 with 8, 1.5e-3 with 16, 1.2e-3 with 32; half as much again, and once more on the shortest."""
    src = torch.stack([matrix(m, n, "gauss", k) for k in range(64)])
    out = torch.full_like(src, float("nan"))
    gtp.gtp_orthogonalize(src, out, workspace(64, m, n))
    for k in range(64):
        want = O.orthogonalize(f64(src[k]))
        assert np.linalg.norm(f64(out[k]) - want) <= bound * np.linalg.norm(want), k
    assert gtp.gtp_wait_timeouts() == 0
