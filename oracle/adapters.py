"""fp64 oracle of low-rank adapters of many requests beside a projection (test infrastructure only).

Rows starts[i] .. starts[i+1] with e = ids[i] >= 0:  y = base + s_e (x D_e^T) U_e^T; for the upstream gradient dy,
dx = dx_base + s_e (dy U_e) D_e, dD_e = sum s_e (dy U_e)^T x, dU_e = sum s_e dy^T (x D_e^T).
"""
from __future__ import annotations

import numpy as np

from .kron import as64


def _requests(N, ids, starts):
    starts = np.arange(N + 1) if starts is None else np.clip(np.asarray(starts), 0, N)
    for i, e in enumerate(np.asarray(ids)):
        if e >= 0 and starts[i + 1] > starts[i]:
            yield slice(int(starts[i]), int(starts[i + 1])), int(e)


def forward(x, base, down, up, ids, starts=None, scales=None):
    """(y, size): size bounds the terms that y is summed from."""
    x, down, up, y = as64(x), as64(down), as64(up), as64(base).copy()
    size = np.abs(y)
    for rows, e in _requests(len(x), ids, starts):
        s = 1.0 if scales is None else float(scales[e])
        y[rows] += s * (x[rows] @ down[e].T) @ up[e].T
        size[rows] += abs(s) * (np.abs(x[rows]) @ np.abs(down[e]).T) @ np.abs(up[e]).T
    return y, size


def backward(x, dy, down, up, ids, starts=None, scales=None, dx_base=None):
    """(dict(dx, ddown, dup), the same of sizes)."""
    x, dy, down, up = as64(x), as64(dy), as64(down), as64(up)
    out = dict(dx=np.zeros_like(x) if dx_base is None else as64(dx_base).copy(), ddown=np.zeros_like(down), dup=np.zeros_like(up))
    size = {k: np.abs(v) for k, v in out.items()}
    for rows, e in _requests(len(x), ids, starts):
        s = 1.0 if scales is None else float(scales[e])
        for o, f in ((out, lambda v: v), (size, np.abs)):
            X, G, D, U, c = f(x[rows]), f(dy[rows]), f(down[e]), f(up[e]), f(s)
            g = c * (G @ U)
            o["dx"][rows] += g @ D
            o["ddown"][e] += g.T @ X
            o["dup"][e] += c * G.T @ (X @ D.T)
    return out, size
