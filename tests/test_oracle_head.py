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


def test_sample_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    pick = lambda u, **kw: head.sample(z, u, **kw)[0]
    assert [pick(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.999)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    assert [pick(u, k=2) for u in (0.0, 0.56, 0.58)] == [1, 1, 3]       # 4/7 of {1, 3}
    assert [pick(u, p=0.65) for u in (0.56, 0.58)] == [1, 3]            # 0.4 + 0.3 >= 0.65
    assert [pick(u, min_p=0.6) for u in (0.56, 0.58)] == [1, 3]         # 0.3 >= 0.6 * 0.4
    assert pick(0.999, p=0.0) == 1 and pick(0.999, min_p=1.0) == 1 and pick(0.9, T=0.0) == 1
    assert head.sample(z, 0.0, k=2)[1] == pytest.approx(np.log(4 / 7))
    # top-p counts the mass that top-k left: 0.4 / 0.7 reaches 0.5 alone
    assert pick(0.999, k=2, p=0.5) == 1


def test_sample_ties_masks_and_refusals():
    z = np.array([1.0, 2.0, 2.0, 2.0, -np.inf])
    assert {head.sample(z, u, k=2)[0] for u in (0.0, 0.49, 0.51, 0.99)} == {1, 2}
    assert {head.sample(z[1:4], u, p=0.5)[0] for u in (0.0, 0.99)} == {0, 1}
    assert head.sample(np.full(4, -np.inf), 0.5)[0] == -1
    assert head.sample(np.array([0.0, np.nan]), 0.5)[0] == -1
    assert head.sample(z, 1.0)[0] == -1 and head.sample(z, 0.5, T=-1.0)[0] == -1
    assert head.sample(np.array([np.inf, 0.0, np.inf]), 0.6)[0] == 2


def test_sample_frequencies():
    rng = np.random.default_rng(8)
    z = rng.normal(size=50)
    u = (np.arange(20000) + 0.5) / 20000
    got = np.bincount([head.sample(z, x)[0] for x in u], minlength=50) / u.size
    assert np.max(np.abs(got - np.exp(z) / np.exp(z).sum())) <= 1 / u.size + 1e-12
