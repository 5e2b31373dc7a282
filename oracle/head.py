"""FP64 reference of the operators around the vocabulary head: the residual +
RMS norm and its gradient, the microscaled formats, the head's product over
them, and the draw of a token.  numpy only, written from the formulas; it
shares no code with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 32
E4M3, E2M1 = "e4m3", "e2m1"


# ---- residual + RMS norm ---------------------------------------------------------

def rms_forward(x, w, residual=None, eps=1e-6, w0=0.0):
    """(y, rstd, h) of rows (M, H)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    with np.errstate(all="ignore"):
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
        y = h * rstd[:, None] * (np.asarray(w, np.float64) + w0)
    return y, rstd, h


def rms_backward(dy, h, w, rstd, dh=None, w0=0.0):
    """(dx, dw) and the sizes (T, S) of the terms added in each, for error bounds."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    g = dy * (np.asarray(w, np.float64) + w0)
    xh = h * r
    dx = r * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    T = np.abs(r) * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
        T = T + np.abs(np.asarray(dh, np.float64))
    return dx, np.sum(dy * xh, axis=0), T, np.sum(np.abs(dy * xh), axis=0)


# ---- microscaled formats ------------------------------------------------------------

def code_values(fmt):
    """Value of every code: 256 of E4M3, 16 of E2M1."""
    n, mb, bias = (256, 3, 7) if fmt == E4M3 else (16, 1, 1)
    out = np.zeros(n)
    for c in range(n):
        mag = c % (n // 2)
        ex, man = mag >> mb, mag & ((1 << mb) - 1)
        if fmt == E4M3 and mag == 127:
            v = np.nan
        elif ex == 0:
            v = man / (1 << mb) * 2.0 ** (1 - bias)
        else:
            v = (1 + man / (1 << mb)) * 2.0 ** (ex - bias)
        out[c] = -v if c >= n // 2 else v
    return out


def vmax(fmt):
    return 448.0 if fmt == E4M3 else 6.0


def scale_bytes(amax, fmt):
    """Least b in 0..254 with amax <= vmax 2^(b - 127); 255 for NaN or infinity."""
    amax = np.asarray(amax, np.float64)
    b = np.full(amax.shape, 255, np.int64)
    for e in range(254, -1, -1):
        b[amax <= vmax(fmt) * 2.0 ** (e - 127)] = e
    b[~np.isfinite(amax)] = 255
    return b


def quantize(x, fmt):
    """(codes (rows, K), scale bytes (rows, K / 32)) of finite or special values."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    b = x.reshape(rows, K // BLOCK, BLOCK)
    with np.errstate(invalid="ignore"):
        sb = scale_bytes(np.max(np.abs(b), axis=2), fmt)
    pos = code_values(fmt)[:(127 if fmt == E4M3 else 8)]
    bad = sb == 255
    a = np.abs(np.where(bad[:, :, None], 0.0, b)) / 2.0 ** (np.where(bad, 127, sb)[:, :, None]
                                                            - 127.0)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    # nearest; a tie goes to the even code
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    neg = np.signbit(b) & ~bad[:, :, None]
    code = code + np.where(neg, 128 if fmt == E4M3 else 8, 0)
    return code.reshape(rows, K).astype(np.uint8), sb.astype(np.uint8)


def pack(codes, fmt):
    return codes if fmt == E4M3 else (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(q, fmt):
    if fmt == E4M3:
        return q
    out = np.empty((q.shape[0], q.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def dequantize(q, scales, fmt):
    v = code_values(fmt)[unpack(q, fmt)]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    return v * np.repeat(s, BLOCK, axis=1)


def step_at(v, s, fmt):
    """Distance of neighbouring values of the grid s * fmt around |v|."""
    mb, emin = (3, -6) if fmt == E4M3 else (1, 0)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(v) / s, 2.0 ** emin)))
    return s * 2.0 ** (e - mb)


# ---- drawing a token -------------------------------------------------------------

def sample(z, u, T=1.0, k=0, p=1.0, min_p=0.0):
    """(token, log-probability) of one row z, by sorting; (-1, nan) without an answer."""
    z = np.asarray(z, np.float64) + 0.0
    V = z.size
    bad = -1, np.nan
    if np.isnan(z).any() or not (T >= 0 and T < np.inf and 0 <= u < 1) or np.isnan(p) or \
            np.isnan(min_p):
        return bad
    m = z.max()
    if m == -np.inf:
        return bad
    if T == 0:
        return int(np.argmax(z)), 0.0
    if m == np.inf:
        w = (z == m).astype(np.float64)
    else:
        w = np.exp((z - m) / np.float64(T))
    order = np.argsort(-z, kind="stable")
    order = order[w[order] >= 0]
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        cum = np.cumsum(w[order])
        n = int(np.searchsorted(cum, np.float64(p) * cum[-1], side="left")) + 1
        order = order[:n]
    keep = np.sort(order[w[order] >= min(np.float64(min_p), 1.0)])
    cum = np.cumsum(w[keep])
    j = int(np.searchsorted(cum, np.float64(u) * cum[-1], side="right"))
    return int(keep[j]), float(np.log(w[keep[j]] / cum[-1]))
