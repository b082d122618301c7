"""Float64 oracle of the orthogonalised optimiser step (the Muon rule): the
momentum's singular values are driven towards 1 by an odd quintic applied
`steps` times, written on the matrix itself (no Gram form)."""
from __future__ import annotations

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def orthogonalise(u: np.ndarray, steps: int = 5, coefs=COEFS, eps: float = 1e-7) -> np.ndarray:
    a, b, c = coefs
    x = u.astype(np.float64)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (np.sqrt((x * x).sum()) + eps)
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def step(master, m, grad, lr, momentum=0.95, nesterov=True, scale=1.0, weight_decay=0.0, eps=1e-7, steps=5, coefs=COEFS):
    """(new master, new m, x)"""
    m = momentum * m.astype(np.float64) + grad
    u = grad + momentum * m if nesterov else m
    x = orthogonalise(u, steps, coefs, eps)
    return (1.0 - lr * weight_decay) * master.astype(np.float64) - lr * scale * x, m, x
