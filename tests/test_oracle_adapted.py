"""The FP64 references of the adapted head's operators on their own: against torch in float64
(autograd and its AdamW), enumeration, and identities.  CPU only."""
import numpy as np
import pytest
import torch

from oracle import adapters, beam, head, step


def rnd(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("shared", ["w", "base", "none"])
def test_adapters_against_autograd(shared):
    M, H, V, n, r = 7, 10, 6, 3, 4
    x, a, b = rnd(M, H, seed=1), rnd(n, r, H, seed=2), rnd(n, V, r, seed=3)
    k, s = np.array([0, 2, -1, 2, 0, 0, 2]), np.array([0.5, 3.0, -1.5])
    w = rnd(V, H, seed=4) if shared == "w" else None
    base = rnd(M, V, seed=5) if shared == "base" else None
    X, A, B = (torch.tensor(t, requires_grad=True) for t in (x, a, b))
    y = torch.zeros((M, V), dtype=torch.float64)
    if w is not None:
        y = X @ torch.tensor(w).T
    if base is not None:
        y = torch.tensor(base)
    rows = [y[i] + (s[k[i]] * (B[k[i]] @ (A[k[i]] @ X[i])) if k[i] >= 0 else 0) for i in range(M)]
    y = torch.stack(rows)
    got, S1, S2 = adapters.forward(x, a, b, k, w, base, s)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-13, atol=1e-13)
    assert (np.abs(got - (base if base is not None else 0)) <= S1 + S2 + 1e-12).all()
    dy = rnd(M, V, seed=6)
    y.backward(torch.tensor(dy))
    (dx, da, db), sums = adapters.backward(dy, x, a, b, k, w, None, s)
    for g, t in ((dx, X), (da, A), (db, B)):
        np.testing.assert_allclose(g, t.grad.numpy(), rtol=1e-12, atol=1e-12)
    assert not da[1].any() and not db[1].any()  # no token has adapter 1
    assert (np.abs(dx) <= sums[0] + sums[1] + 1e-12).all()
    assert (np.abs(da) <= sums[2] + 1e-12).all() and (np.abs(db) <= sums[3] + 1e-12).all()


@pytest.mark.parametrize("betas,eps,wd", [((0.9, 0.999), 1e-8, 0.01), ((0.5, 0.8), 1e-3, 0.3)])
def test_adamw_against_torch(betas, eps, wd):
    p = torch.tensor(rnd(50, seed=1), requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.02, betas=betas, eps=eps, weight_decay=wd)
    q, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 8):
        g = rnd(50, seed=10 + t)
        p.grad = torch.tensor(g)
        opt.step()
        q, m, v = step.adamw(q, g, m, v, 0.02, t, *betas, eps, wd)
        np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_moments32_rounds_each_operation():
    g, m, v = (rnd(1000, seed=i).astype(np.float32) for i in (1, 2, 3))
    v = v * v
    a, b = step.moments32(g, 0.5, m, v, 0.9, 0.999)
    _, m1, v1 = step.adamw(0 * g, g * 0.5, m, v, 0.0, 1, 0.9, 0.999)
    u = 2.0 ** -24
    assert (np.abs(a - m1) <= 5 * u * (0.9 * np.abs(m) + 0.05 * np.abs(g))).all()
    assert (np.abs(b - v1) <= 8 * u * v1).all()


def test_mix_is_one_to_one_and_even():
    n = 1 << 16
    x = np.arange(n, dtype=np.uint64) * np.uint64(65537)
    assert len(np.unique(step.mix(x))) == n
    bits = step.random_bits(np.arange(n), 3, 5)
    for half in (bits & np.uint64(65535), bits >> np.uint64(16)):
        # 64 cells of 1024 expected: within six standard deviations
        count = np.bincount((half >> np.uint64(10)).astype(int), minlength=64)
        assert (np.abs(count - 1024) <= 6 * np.sqrt(1024)).all()
    # other places, steps and seeds give other numbers
    for args in ((np.arange(n) + (1 << 32), 3, 5), (np.arange(n), 3, 6), (np.arange(n), 1 << 33, 5)):
        same = (step.random_bits(*args) == bits).mean()
        assert same < 1e-3


def test_round_random():
    x = np.linspace(-448, 448, 32 * 40)
    x[::7] = 0
    for r in (0, 1, 30000, 65535):
        code, sc = step.round_random(x, np.full(x.shape, r), False)
        got = head.dequantize(code.reshape(1, -1), sc.reshape(1, -1), "e4m3").reshape(-1)
        s = np.repeat(2.0 ** (sc.astype(float) - 127), 32)
        place = np.maximum(2.0 ** np.floor(np.log2(np.maximum(np.abs(x) / s, 1e-30))), 2.0 ** -6)
        h = place / 8 * s
        assert (np.abs(got - x) < h).all() and (got[x == 0] == 0).all()
        exact = np.abs(np.round(x / h) * h - x) < 1e-13
        assert (np.abs(got - x)[exact] < 1e-12).all()
        if r == 65535:  # hardly anything goes up
            assert (np.abs(got) <= np.abs(x) + 2.0 ** -15 * h).all()
    tiny = np.zeros(32)
    tiny[0], tiny[1], tiny[2] = 400.0, 1e-9, 0.0
    for keep, want in ((False, 0), (True, 1)):
        assert step.round_random(tiny, np.full(32, 65535), keep)[0][:3].tolist()[1:] == [want, 0]
    bad = np.ones(64)
    bad[3] = np.nan
    code, sc = step.round_random(bad, np.zeros(64), False)
    assert sc.tolist()[0] == 255 and not code[:32].any() and sc[1] != 255


def test_beam_against_enumeration():
    K, V = 3, 5
    z, s = rnd(K, V, seed=1), np.array([-1.0, -0.5, -3.0])
    z[1, 2] = -np.inf
    p = torch.log_softmax(torch.tensor(z), 1).numpy()
    every = sorted((-(s[k] + p[k, v]), k, v) for k in range(K) for v in range(V)
                   if np.isfinite(z[k, v]))
    score, par, tok = beam.step(z, s, 20)
    assert list(zip(par[:14], tok[:14])) == [(k, v) for _, k, v in every]
    np.testing.assert_allclose(score[:14], [-c for c, _, _ in every], rtol=1e-12)
    assert (par[14:] == -1).all() and (tok[14:] == -1).all() and (score[14:] == -np.inf).all()
    ended = [False, True, False]
    score, par, tok = beam.step(z, s, 12, ended, 4)
    assert (par == 1).sum() == 1 and tok[par == 1][0] == 4 and score[par == 1][0] == -0.5
    # ties: the lower beam, then the lower token
    _, par, tok = beam.step(np.zeros((2, 3)), np.zeros(2), 6)
    assert par.tolist() == [0, 0, 0, 1, 1, 1] and tok.tolist() == [0, 1, 2, 0, 1, 2]
