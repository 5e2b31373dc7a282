"""The FP64 reference of the operators around the head, pinned on its own:
gradients against central differences, the formats against their definitions."""
import numpy as np
import pytest

from oracle import head


@pytest.mark.parametrize("with_res", [False, True])
def test_rms_backward_matches_differences(with_res):
    rng = np.random.default_rng(5)
    M, H, w0, eps = 3, 7, 1.0, 1e-3
    x, w = rng.normal(size=(M, H)), 0.3 * rng.normal(size=H)
    res = rng.normal(size=(M, H)) if with_res else None
    cy, ch = rng.normal(size=(M, H)), rng.normal(size=(M, H))

    def f(x, w):
        y, _, h = head.rms_forward(x, w, res, eps, w0)
        return np.sum(cy * y) + (np.sum(ch * h) if with_res else 0.0)
    _, rstd, h = head.rms_forward(x, w, res, eps, w0)
    dx, dw, _, _ = head.rms_backward(cy, h, w, rstd, ch if with_res else None, w0)
    d = 1e-5
    for i in range(M):
        for j in range(H):
            e = np.zeros_like(x)
            e[i, j] = d
            assert abs((f(x + e, w) - f(x - e, w)) / (2 * d) - dx[i, j]) < 1e-7
    for j in range(H):
        e = np.zeros_like(w)
        e[j] = d
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * d) - dw[j]) < 1e-7


def test_format_grids():
    v = head.code_values("e2m1")
    assert v[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and v[15] == -6
    v = head.code_values("e4m3")
    assert v[0x7E] == 448 and np.isnan(v[0x7F]) and v[1] == 2.0 ** -9 and v[0x38] == 1
    assert np.all(np.diff(v[:127]) > 0)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_quantize_is_nearest_and_never_clips(fmt):
    rng = np.random.default_rng(6)
    x = rng.normal(size=(20, 96)) * 2.0 ** rng.integers(-20, 20, size=(20, 1))
    q, s = head.quantize(x, fmt)
    q = head.pack(q, fmt)
    v = head.dequantize(q, s, fmt)
    sc = np.repeat(2.0 ** (s.astype(float) - 127), 32, axis=1)
    assert np.all(np.abs(x) <= head.vmax(fmt) * sc)
    assert np.all(np.abs(v - x) <= head.step_at(x, sc, fmt) / 2)
    # least scale: one step less would clip
    assert np.all(np.max(np.abs(x).reshape(20, 3, 32), 2) > head.vmax(fmt) * 2.0 **
                  (s.astype(float) - 128))


def test_quantize_special_blocks():
    x = np.zeros((1, 96))
    x[0, 40], x[0, 70] = np.nan, np.inf
    q, s = head.quantize(x, "e2m1")
    assert s.tolist() == [[0, 255, 255]] and not q.any()
