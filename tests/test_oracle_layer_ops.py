"""The oracles of the embedding, the norm and the orthogonalised update against something other than themselves."""
import numpy as np
import pytest
import torch

from oracle import embedding as E
from oracle import orthogonalize as O
from oracle import rmsnorm as N


def test_embedding_is_torch_s_within_the_shard():
    rng = np.random.default_rng(0)
    table = rng.normal(size=(10, 6))
    ids = np.array([3, 12, 5, 5, 4, 13, -1, 3])
    want = torch.nn.functional.embedding(torch.tensor([0, 9, 2, 2, 1, 0, 0, 0]), torch.tensor(table)).numpy() * 2.5
    want[[5, 6]] = 0  # 13 and -1 are no rows of a shard of ten from 3 on
    got = E.lookup(ids, table, 3, 2.5)
    assert np.allclose(got, want, rtol=1e-15)
    t = torch.tensor(table, requires_grad=True)
    dout = rng.normal(size=(8, 6))
    dout[[5, 6]] = 0
    (torch.nn.functional.embedding(torch.tensor([0, 9, 2, 2, 1, 0, 0, 0]), t) * 2.5 * torch.tensor(dout)).sum().backward()
    grad, mass, n = E.gradient(ids, dout, 10, 3, 2.5)
    assert np.allclose(grad, t.grad.numpy(), rtol=1e-14)
    assert n.tolist() == [2, 1, 2, 0, 0, 0, 0, 0, 0, 1] and np.all(mass >= np.abs(grad) - 1e-15)


@pytest.mark.parametrize("dsum", [False, True])
def test_norm_is_autograd_s(dsum):
    rng = np.random.default_rng(1)
    s, w, dy, ds = rng.normal(size=(5, 12)), rng.normal(size=12), rng.normal(size=(5, 12)), rng.normal(size=(5, 12))
    ts, tw = torch.tensor(s, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = torch.nn.functional.rms_norm(ts, (12,), tw, 1e-5)
    rstd, got = N.forward(s, w, 1e-5)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-13)
    ((y * torch.tensor(dy)).sum() + (ts * torch.tensor(ds)).sum() * dsum).backward()
    dx, dw = N.gradient(dy, s, rstd, w, ds if dsum else None)
    assert np.allclose(dx, ts.grad.numpy(), rtol=1e-12) and np.allclose(dw, tw.grad.numpy(), rtol=1e-12)


@pytest.mark.parametrize("shape", [(7, 19), (19, 7), (8, 8)])
def test_iteration_acts_on_singular_values_alone(shape):
    rng = np.random.default_rng(2)
    G = rng.normal(size=shape)
    U, S, V = np.linalg.svd(G, full_matrices=False)
    s = S / np.linalg.norm(G)
    a, b, c = (float(np.float32(v)) for v in O.COEFFICIENTS)
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    assert np.allclose(O.orthogonalize(G), (U * s) @ V, atol=1e-12)
    assert not O.orthogonalize(np.zeros(shape)).any()


def test_step_without_momentum_moves_along_the_orthogonal_update():
    rng = np.random.default_rng(3)
    g, p = rng.normal(size=(4, 9)), rng.normal(size=(4, 9))
    m, q = O.step(g, np.zeros((4, 9)), p, 0.0, 0.1, 0.5, 2.0)
    assert np.allclose(m, g) and np.allclose(q, p * 0.95 - 0.2 * O.orthogonalize(g))
    m, q = O.step(g, g, p, 0.75, 0.1, 0.0, 1.0, nesterov=False)
    assert np.allclose(m, g) and np.allclose(q, p - 0.1 * O.orthogonalize(3 * g))
