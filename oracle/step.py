"""FP64 reference of the optimizer step and the gradients' norm, and the FP32
arithmetic of the 8-bit states bit by bit.  numpy only, written from the
formulas; it shares no code with the library."""
from __future__ import annotations

import numpy as np

from . import head

WORD = np.uint64(0xFFFFFFFF)


def adamw(p, g, m, v, lr, step, b1=0.9, b2=0.999, eps=1e-8, wd=0.01):
    """(p, m, v) after one step, in FP64."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    with np.errstate(all="ignore"):
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
        return p - lr * wd * p - lr * mh / (np.sqrt(vh) + eps), m, v


def moments32(g, scale, m, v, b1, b2):
    """(m, v) in FP32, every operation rounded by itself."""
    f = np.float32
    with np.errstate(all="ignore"):
        g = g.astype(f) * f(scale)
        m = m.astype(f) * f(b1) + g * f(1.0 - b1)
        v = v.astype(f) * f(b2) + (g * g) * f(1.0 - b2)
    return m, v


def mix(x):
    x = (x ^ (x >> np.uint64(16))) * np.uint64(0x9E3779B9) & WORD
    x = (x ^ (x >> np.uint64(15))) * np.uint64(0x6A09E667) & WORD
    return x ^ (x >> np.uint64(16))


def random_bits(places, seed, step):
    """32 bits for each flat place."""
    i = np.asarray(places, np.uint64)
    one = lambda t: np.array([t], np.uint64)
    k = mix(one(seed & 0xFFFFFFFF) ^ mix(one(seed >> 32)))
    k = mix((k + one(step)) & WORD)
    return mix((i & WORD) ^ mix((k + (i >> np.uint64(32))) & WORD))


def round_random(x, r16, keep):
    """FP32 values (a multiple of 32) to E4M3 codes and scale bytes, up where the part below a
    code's last place, in 65536ths, exceeds r16."""
    b = np.asarray(x, np.float64).reshape(-1, 32)
    r = np.asarray(r16, np.float64).reshape(-1, 32)
    grid = head.code_values("e4m3")[:127]  # 0 .. 448
    code = np.zeros(b.shape, np.uint8)
    scales = np.zeros(len(b), np.uint8)
    for i, row in enumerate(b):
        if not np.isfinite(row).all():
            scales[i] = 255
            continue
        e = -127
        while np.abs(row).max() > 448 * 2.0 ** e:
            e += 1
        a = np.abs(row) / 2.0 ** e
        lo = np.searchsorted(grid, a, side="right") - 1
        hi = np.minimum(lo + 1, 126)
        part = np.where(hi > lo, (a - grid[lo]) / np.where(hi > lo, grid[hi] - grid[lo], 1), 0)
        c = np.where(part * 65536 > r[i], hi, lo)
        if keep:
            c = np.where((a > 0) & (c == 0), 1, c)
        code[i] = c | np.where(row < 0, 128, 0)
        scales[i] = e + 127
    return code.reshape(-1), scales
