"""Newton-Schulz orthogonalisation and the step on it (oracle; test infrastructure): float64, from the definitions."""
from __future__ import annotations

import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(G, steps: int = 5, coefficients=COEFFICIENTS) -> np.ndarray:
    a, b, c = (float(np.float32(v)) for v in coefficients)
    X = np.asarray(G, np.float64)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    norm = np.linalg.norm(X)
    X = X / norm if norm > 0 else X
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.T if tall else X


def step(grad, momentum, master, mu, lr, decay, scale, nesterov=True, **how):
    """(momentum, master) after the step."""
    g, m, p = (np.asarray(a, np.float64) for a in (grad, momentum, master))
    m = mu * m + (1 - mu) * g
    u = mu * m + (1 - mu) * g if nesterov else m
    return m, p * (1 - lr * decay) - lr * scale * orthogonalize(u, **how)
