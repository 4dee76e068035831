"""fp64 oracle of the gated Kronecker block, through the materialised weights (test infrastructure only).

  g = x W_0 + b_0,  u = x W_1 + b_1,  y = act(g) o u,  W_f = sum_i kron(S_f o A_fi, B_fi)
  dg = dy u act'(g),  du = dy act(g),  dx = dg W_0^T + du W_1^T, and each projection's parameter
gradients are the layer's (kron.backward) for its own upstream gradient.
"""
from __future__ import annotations

import math

import numpy as np

from . import kron
from .kron import as64

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(kind, v):
    """(act(v), act'(v))"""
    v = as64(v)
    if kind == "silu":
        s = 1 / (1 + np.exp(-v))
        return v * s, s + v * s * (1 - s)
    if kind == "gelu":
        c = 0.5 * (1 + _erf(v / math.sqrt(2)))
        return v * c, c + v * np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = np.tanh(a * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * a * (1 + 3 * 0.044715 * v * v)
    return np.maximum(v, 0), (v > 0).astype(np.float64)


def _half(t, f):
    return None if t is None else t[f]


def project(x, S, A, B, bias):
    """The two projections' outputs g and u."""
    return [as64(x) @ kron.weight(_half(S, f), A[f], B[f]) + (0 if bias is None else as64(bias[f])) for f in range(2)]


def forward(x, S, A, B, bias, act):
    g, u = project(x, S, A, B, bias)
    return activation(act, g)[0] * u


def backward(x, S, A, B, bias, dy, act):
    g, u = project(x, S, A, B, bias)
    a, da = activation(act, g)
    d = [as64(dy) * u * da, as64(dy) * a]
    got = [kron.backward(x, _half(S, f), A[f], B[f], d[f]) for f in range(2)]
    out = {k: np.stack([h[k] for h in got]) for k in ("dA", "dB", "dbias")}
    out["dS"] = None if S is None else np.stack([h["dS"] for h in got])
    out["dx"] = got[0]["dx"] + got[1]["dx"]
    return out
