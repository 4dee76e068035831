"""fp64 oracle of the orthogonalised (Muon) update (test infrastructure only).

m = mu m + g; u = g + mu m or m; X = u / (|u|_F + eps); steps times X = a X + (b A + c A^2) X with A = X X^T (a Newton-Schulz
step on the quintic of the singular values); param = param (1 - lr wd) - lr scale X.  `dtype` computes the same in
another precision, `part` rounds each product's operands (a model of the roundings, for tolerances).
"""
from __future__ import annotations

import numpy as np

COEFFS = (3.4445, -4.7750, 2.0315)


def orthogonalise(u, steps=5, coeffs=COEFFS, eps=1e-7, dtype=np.float64, part=lambda v: v):
    a, b, c = (dtype(v) for v in coeffs)
    X = np.asarray(u, dtype)
    tall = X.shape[0] > X.shape[1]
    X = X.T if tall else X
    X = X / dtype(np.sqrt((X.astype(np.float64) ** 2).sum()) + eps)
    for _ in range(steps):
        X = part(X)
        A = part(X @ X.T)
        P = part(a * np.eye(len(A), dtype=dtype) + b * A + c * (A @ A))
        X = P @ X
    return X.T if tall else X


def step(param, grad, m, lr, mu=0.95, nesterov=True, wd=0.0, scale=1.0, **kw):
    """(param, m, the orthogonalised matrix) of one matrix."""
    param, grad, m = (np.asarray(v, np.float64) for v in (param, grad, m))
    m = mu * m + grad
    o = orthogonalise(grad + mu * m if nesterov else m, **kw)
    return param * (1 - lr * wd) - lr * scale * o, m, o
