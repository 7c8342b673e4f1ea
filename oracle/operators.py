"""fp64 embedding, layer norm and distillation loss, with their gradients, from the formulas: the plain statement the
CUDA kernels are compared with. Test infrastructure only."""
from __future__ import annotations

import numpy as np


def embedding_forward(ids, table, scale):
    table = np.asarray(table, np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for i, v in enumerate(ids):
        if 0 <= v < table.shape[0]:
            out[i] = scale * table[v]
    return out


def embedding_backward(ids, dout, V, scale, padding_idx=-1):
    """Returns (gradient, occurrences of each id, sum of |scale * dout| for each element)."""
    D = dout.shape[1]
    g, mag, count = np.zeros((V, D)), np.zeros((V, D)), np.zeros(V, np.int64)
    for v, row in zip(ids, np.asarray(dout, np.float64)):
        if 0 <= v < V and v != padding_idx:
            g[v] += scale * row
            mag[v] += abs(scale) * np.abs(row)
            count[v] += 1
    return g, count, mag


def layernorm_forward(x, w, b, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * (1.0 if w is None else w) + (0.0 if b is None else b)
    return y, mean, rstd


def layernorm_backward(dy, x, w, mean, rstd):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    xh = (x - np.asarray(mean)[:, None]) * np.asarray(rstd)[:, None]
    g = dy * (1.0 if w is None else w)
    dx = np.asarray(rstd)[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def distill(z, t_idx, t_val, T, weights=None):
    """Returns a dict: losses, stats (N, 2), dlogits (the gradient of the losses' sum), and p, q (N, V) of live rows."""
    z = np.asarray(z, np.float64)
    t = np.asarray(t_val, np.float64)
    N, V = z.shape
    w = np.ones(N) if weights is None else np.asarray(weights, np.float64)
    losses, stats, dz = np.zeros(N), np.zeros((N, 2)), np.zeros((N, V))
    P, Q = np.zeros((N, V)), np.zeros((N, V))
    for i in range(N):
        ok = [k for k in range(t.shape[1]) if 0 <= t_idx[i, k] < V and t[i, k] != -np.inf]
        if w[i] == 0 or not ok:
            continue
        idx, tv = np.asarray(t_idx[i])[ok], t[i][ok] / T
        lq = tv - tv.max()
        lq = lq - np.log(np.exp(lq).sum())
        q = np.exp(lq)
        m = z[i].max()
        with np.errstate(invalid="ignore"):
            x = (z[i] - m) / T
        l = np.log(np.exp(x).sum())
        lp = x - l
        kl = sum(qk * (lqk - lp[j]) for qk, lqk, j in zip(q, lq, idx) if qk > 0)
        losses[i] = w[i] * T * T * kl
        stats[i] = m, l
        P[i] = np.exp(lp)
        np.add.at(Q[i], idx, q)
        dz[i] = w[i] * T * (P[i] - Q[i])
    return {"losses": losses, "stats": stats, "dlogits": dz, "p": P, "q": Q}
