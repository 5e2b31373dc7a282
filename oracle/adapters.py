"""FP64 reference of the low-rank adapters, token by token's adapter.  numpy only, written from
the formulas; it shares no code with the library."""
from __future__ import annotations

import numpy as np


def _on(adapter, scale, n):
    k = np.asarray(adapter)
    s = np.ones(n) if scale is None else np.asarray(scale, np.float64)
    return [(i, s[i], np.flatnonzero(k == i)) for i in range(n)]


def forward(x, a, b, adapter, w=None, base=None, scale=None):
    """(y, S1, S2): y and the sums of the absolute terms of the shared and the adapters' part."""
    x, a, b = (np.asarray(t, np.float64) for t in (x, a, b))
    M, V = x.shape[0], b.shape[1]
    y, S1, S2 = np.zeros((M, V)), np.zeros((M, V)), np.zeros((M, V))
    with np.errstate(all="ignore"):
        if w is not None:
            w = np.asarray(w, np.float64)
            y, S1 = x @ w.T, np.abs(x) @ np.abs(w).T
        elif base is not None:
            y = np.array(base, np.float64)
        for k, s, rows in _on(adapter, scale, a.shape[0]):
            if len(rows):
                y[rows] += s * ((x[rows] @ a[k].T) @ b[k].T)
                S2[rows] = abs(s) * ((np.abs(x[rows]) @ np.abs(a[k]).T) @ np.abs(b[k]).T)
    return y, S1, S2


def backward(dy, x, a, b, adapter, w=None, dx_base=None, scale=None):
    """(dx, da, db) and the sums of the absolute terms (S1, S2 of dx, Sa, Sb)."""
    dy, x, a, b = (np.asarray(t, np.float64) for t in (dy, x, a, b))
    dx, S1, S2 = (np.zeros(x.shape) for _ in range(3))
    da, Sa, db, Sb = np.zeros(a.shape), np.zeros(a.shape), np.zeros(b.shape), np.zeros(b.shape)
    if w is not None:
        w = np.asarray(w, np.float64)
        dx, S1 = dy @ w, np.abs(dy) @ np.abs(w)
    elif dx_base is not None:
        dx = np.array(dx_base, np.float64)
    for k, s, rows in _on(adapter, scale, a.shape[0]):
        if not len(rows):
            continue
        d, t = dy[rows], x[rows]
        ds, sx = s * (d @ b[k]), s * (t @ a[k].T)
        Ds, Sx = abs(s) * (np.abs(d) @ np.abs(b[k])), abs(s) * (np.abs(t) @ np.abs(a[k]).T)
        dx[rows] += ds @ a[k]
        S2[rows] = Ds @ np.abs(a[k])
        da[k], Sa[k] = ds.T @ t, Ds.T @ np.abs(t)
        db[k], Sb[k] = d.T @ sx, np.abs(d).T @ Sx
    return (dx, da, db), (S1, S2, Sa, Sb)
