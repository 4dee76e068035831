"""fp64 oracle of a teacher's top logits and of the distillation loss (test infrastructure only).

With T the temperature and q = softmax(z / T) of a student's row z, ids and t the teacher's kept
tokens and logits:
  without the teacher's lse:  p = softmax(t / T),  KD = sum_j p_j (log p_j - log q[id_j])
  with it:  p_j = exp(t_j / T - lse),  p_t = max(0, 1 - sum p),  q_t = the mass of q off the kept
            tokens,  KD = sum_j p_j (log p_j - log q[id_j]) + p_t (log p_t - log q_t)
  loss = sum_n w_n (alpha T^2 KD_n + (1 - alpha) (logsumexp(z_n) - z_n[label_n]))
The gradient goes through the log-softmax: for L(log q), dL/dz = (g - q sum(g)) / T with
g = dL/dlog q.
"""
from __future__ import annotations

import numpy as np

from .kron import as64


def topk(z, k, T=1.0):
    """(ids, values, lse): the k largest of each row, equal values by the lower token."""
    z = as64(z)
    ids = np.stack([np.lexsort((np.arange(z.shape[1]), -row))[:k] for row in z]) if len(z) else np.zeros((0, k), int)
    vals = np.take_along_axis(z, ids, 1)
    m = z.max(1, keepdims=True) if len(z) else np.zeros((0, 1))
    lse = (m / T + np.log(np.exp((z - m) / T).sum(1, keepdims=True)))[:, 0]
    return ids, vals, lse


def _log_softmax(y):
    y = y - y.max()
    return y - np.log(np.exp(y).sum())


def loss_and_grad(z, ids, t, lse=None, labels=None, weights=None, T=1.0, alpha=1.0):
    """(loss, dz, scale, lscale): scale bounds the terms that each gradient is the difference of and
    lscale those of the loss (what relative roundings act on)."""
    z = as64(z)
    N, V = z.shape
    w = np.full(N, 1.0 / max(N, 1)) if weights is None else as64(weights)
    dz, scale = np.zeros((N, V)), np.zeros((N, V))
    loss, lscale = 0.0, 0.0
    for n in range(N):
        if w[n] == 0:
            continue
        if alpha > 0:
            slot = [j for j in range(ids.shape[1]) if ids[n, j] >= 0]
            idn, tn = np.asarray(ids[n])[slot].astype(int), as64(t[n])[slot] / T
            logq = _log_softmax(z[n] / T)
            q = np.exp(logq)
            g, gs = np.zeros(V), np.zeros(V)
            kd = ks = 0.0
            if lse is None:
                live = tn > -np.inf
                logp = np.full(tn.shape, -np.inf)
                if live.any():
                    logp[live] = _log_softmax(tn[live])
            else:
                logp = tn - float(as64(lse)[n])
            p = np.exp(logp)
            for j in range(len(idn)):
                if p[j] > 0:
                    kd += p[j] * (logp[j] - logq[idn[j]])
                    ks += p[j] * (abs(logp[j]) + abs(logq[idn[j]]) + 1)
                g[idn[j]] -= p[j]
                gs[idn[j]] += p[j]
            if lse is not None:
                pt = max(0.0, 1.0 - p.sum())
                off = np.ones(V, bool)
                off[idn] = False
                if pt > 0 and off.any():
                    qt = q[off].sum()
                    kd += pt * (np.log(pt) - np.log(qt))
                    ks += pt * (abs(np.log(pt)) + abs(np.log(qt)) + 1)
                    g[off] -= pt / qt * q[off]
                    gs[off] += pt / qt * q[off]
            dz[n] += alpha * T * (g - q * g.sum())
            scale[n] += alpha * T * (gs + q * gs.sum())
            loss += w[n] * alpha * T * T * kd
            lscale += w[n] * alpha * T * T * ks
        if alpha < 1:
            lq = _log_softmax(z[n])
            g = np.exp(lq)
            s = g.copy()
            g[labels[n]] -= 1
            s[labels[n]] += 1
            dz[n] += (1 - alpha) * g
            scale[n] += (1 - alpha) * s
            loss -= w[n] * (1 - alpha) * lq[labels[n]]
            lscale += w[n] * (1 - alpha) * (abs(lq[labels[n]]) + 1)
        dz[n] *= w[n]
        scale[n] *= abs(w[n])
    return loss, dz, scale, lscale
