"""Plain CPU oracle, in fp64, for the operators around a shared projection: rows sorted by id, the adapters of many
requests and their gradients, the layer norm and its gradient."""
from __future__ import annotations

import numpy as np


def route(ids, n):
    """(order, offsets): the rows of each id in ascending order, those without one behind them."""
    rows = [[] for _ in range(n + 1)]
    for m, i in enumerate(np.asarray(ids).tolist()):
        rows[i if 0 <= i < n else n].append(m)
    offsets = np.cumsum([0] + [len(r) for r in rows[:n]])
    return np.array([m for r in rows for m in r], np.int32), offsets.astype(np.int32)


def layernorm(h, w, b, eps):
    """(y, mean, rstd) of h [M][H] (the residual already added and rounded)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    mean = np.mean(h, 1)
    d = h - mean[:, None]
    rstd = 1.0 / np.sqrt(np.mean(d * d, 1) + eps)
    y = d * rstd[:, None] * w
    return (y if b is None else y + np.asarray(b, np.float64)), mean, rstd


def layernorm_grad(dy, h, w, mean, rstd, dh=None):
    """(dx, dw, db)."""
    dy, h, w, mean, rstd = (np.asarray(t, np.float64) for t in (dy, h, w, mean, rstd))
    xhat = (h - mean[:, None]) * rstd[:, None]
    u = dy * w
    dx = rstd[:, None] * (u - np.mean(u, 1, keepdims=True) - xhat * np.mean(u * xhat, 1, keepdims=True))
    return (dx if dh is None else dx + np.asarray(dh, np.float64)), np.sum(dy * xhat, 0), np.sum(dy, 0)


def _listed(order, offsets, a, M):
    """The rows of adapter a."""
    rows = np.arange(M) if order is None else np.asarray(order)
    return rows[offsets[a]:offsets[a + 1]]


def adapters_fwd(x, l1, l2, s, order, offsets, base):
    """(y, t, S, Q, R): the outputs for listed rows (others: base, or 0 without one, and t = 0); S the sum of the
    magnitudes of the terms of s T L2, Q the same of X L1, and R what Q becomes in Y."""
    x, l1, l2, s = (np.asarray(v, np.float64) for v in (x, l1, l2, s))
    M, n, r, o = x.shape[0], l1.shape[0], l1.shape[2], l2.shape[2]
    y = np.zeros((M, o)) if base is None else np.array(base, np.float64)
    t, S, Q, R = np.zeros((M, r)), np.zeros((M, o)), np.zeros((M, r)), np.zeros((M, o))
    for a in range(n):
        rows = _listed(order, offsets, a, M)
        t[rows] = x[rows] @ l1[a]
        Q[rows] = np.abs(x[rows]) @ np.abs(l1[a])
        y[rows] += s[a] * (t[rows] @ l2[a])
        S[rows] = abs(s[a]) * (np.abs(t[rows]) @ np.abs(l2[a]))
        R[rows] = abs(s[a]) * (Q[rows] @ np.abs(l2[a]))
    return y, t, S, Q, R


def adapters_bwd(dy, x, t, l1, l2, s, order, offsets, base):
    """(dx, dl1, dl2), each with the sum of the magnitudes of its terms (G's own terms in the first two)."""
    dy, x, t, l1, l2, s = (np.asarray(v, np.float64) for v in (dy, x, t, l1, l2, s))
    M, n, h, r, o = x.shape[0], l1.shape[0], l1.shape[1], l1.shape[2], l2.shape[2]
    dx = np.zeros((M, h)) if base is None else np.array(base, np.float64)
    Sx, dl1, S1, dl2, S2 = np.zeros((M, h)), np.zeros((n, h, r)), np.zeros((n, h, r)), np.zeros((n, r, o)), \
        np.zeros((n, r, o))
    for a in range(n):
        rows = _listed(order, offsets, a, M)
        g = s[a] * (dy[rows] @ l2[a].T)
        Sg = abs(s[a]) * (np.abs(dy[rows]) @ np.abs(l2[a]).T)
        dl2[a] = s[a] * (t[rows].T @ dy[rows])
        S2[a] = abs(s[a]) * (np.abs(t[rows]).T @ np.abs(dy[rows]))
        dl1[a] = x[rows].T @ g
        S1[a] = np.abs(x[rows]).T @ Sg
        dx[rows] += g @ l1[a].T
        Sx[rows] = Sg @ np.abs(l1[a]).T
    return (dx, Sx), (dl1, S1), (dl2, S2)
