"""FP64 reference of a beam search step.  numpy only, written from the formulas; it shares
no code with the library."""
from __future__ import annotations

import numpy as np


def step(z, scores, n_out, ended=None, end_token=0):
    """(score, parent, token) of one request: z (K, V), scores (K); all candidates formed and
    sorted by (value down, beam up, token up)."""
    z, scores = np.asarray(z, np.float64), np.asarray(scores, np.float64)
    K, V = z.shape
    val, par, tok = [], [], []
    for k in range(K):
        if not np.isfinite(scores[k]):
            continue
        if ended is not None and ended[k]:
            v, t = np.array([scores[k]]), np.array([end_token])
        else:
            m = z[k].max()
            if not np.isfinite(m) or np.isnan(z[k]).any():
                continue
            lse = m + np.log(np.exp(z[k] - m).sum())
            t = np.flatnonzero(z[k] > -np.inf)
            v = scores[k] + (z[k][t] - lse)
        val.append(v)
        par.append(np.full(len(t), k))
        tok.append(t)
    out = (np.full(n_out, -np.inf), np.full(n_out, -1), np.full(n_out, -1))
    if val:
        val, par, tok = (np.concatenate(a) for a in (val, par, tok))
        best = np.lexsort((tok, par, -val))[:n_out]
        for o, a in zip(out, (val, par, tok)):
            o[:len(best)] = a[best]
    return out
