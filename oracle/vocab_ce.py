"""fp64 oracle of the cross-entropy of a large vocabulary from the hidden states (test infrastructure only).

z = h W^T, nll_n = logsumexp(z_n) - z_n[label_n], loss = sum_n w_n nll_n over the rows of nonzero weight;
dz = w (softmax(z) - onehot), dh = dz W, dW = dz^T h.
"""
from __future__ import annotations

import numpy as np

from .kron import as64


def forward_backward(h, W, labels, weights=None, gout=1.0):
    """dict(loss, nll, dh, dW) and the sizes that roundings act on: zs = |h| |W|^T (the largest of each row), p the
    probabilities, w the weights."""
    h, W = as64(h), as64(W)
    N, V = h.shape[0], W.shape[0]
    w = np.full(N, 1.0 / max(N, 1)) if weights is None else as64(weights)
    used = np.flatnonzero(w != 0)
    nll, dh, dW = np.zeros(N), np.zeros_like(h), np.zeros_like(W)
    x = h[used]
    z = x @ W.T
    m = z.max(1, keepdims=True) if len(used) else np.zeros((0, 1))
    e = np.exp(z - m)
    total = e.sum(1, keepdims=True)
    lab = np.asarray(labels)[used]
    row = np.arange(len(used))
    nll[used] = (m + np.log(total))[:, 0] - z[row, lab]
    p = e / total
    dz = p.copy()
    dz[row, lab] -= 1
    dz *= (w[used] * gout)[:, None]
    dh[used] = dz @ W
    dW += dz.T @ x
    size = np.abs(x) @ np.abs(W).T
    return dict(loss=float((w * nll).sum()), nll=nll, dh=dh, dW=dW, used=used, x=x, W=W, p=p, dz=dz, w=w, z=z,
                zs=size.max(1) if len(used) else np.zeros(0))
