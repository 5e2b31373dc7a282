"""ce_sample against the FP64 reference that sorts.  Tokens are equal; logprob
is off by its own rounding (u |ref|) and by the weights' rounding to 2^-44 of
the largest: at most V 2^-45 in the sum, which is at least 1."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, U, assert_within, f64
from oracle import head

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
FMAX = float(np.finfo(np.float32).max)


def t32(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def run(z, u, T=None, k=None, p=None, mp=None):
    """z (..., V); the rest lists per row."""
    ki = None if k is None else torch.tensor(k, dtype=torch.int32, device="cuda")
    tok, lp = vce.ce_sample(z, t32(u), None if T is None else t32(T), ki,
                            None if p is None else t32(p), None if mp is None else t32(mp),
                            with_logprob=True)
    zz = f64(z).reshape(-1, z.shape[-1])
    f = lambda a, i, off: off if a is None else float(np.float32(a[i]))
    ref = [head.sample(zz[i], f(u, i, 0), f(T, i, 1.0), 0 if k is None else k[i], f(p, i, 1.0),
                       f(mp, i, 0.0)) for i in range(zz.shape[0])]
    got = tok.reshape(-1).tolist()
    want = [a for a, _ in ref]
    assert got == want, [(i, g, w) for i, (g, w) in enumerate(zip(got, want)) if g != w][:5]
    rl = np.array([b for _, b in ref])
    assert_within(f64(lp).reshape(-1), rl, U * np.abs(rl) + zz.shape[1] * 2.0 ** -45 + 1e-15,
                  "logprob")
    return tok


def normal(N, V, dtype, seed, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((N, V), generator=g) * sigma).to(DT[dtype]).cuda()


def params(N, seed):
    r = np.random.default_rng(seed)
    return dict(u=r.random(N, dtype=np.float32).tolist(),
                T=r.choice([0.0, 0.3, 0.7, 1.0, 1.0, 2.0], N).tolist(),
                k=r.choice([0, 0, 1, 2, 40, 1000, 5000, 10 ** 6], N).tolist(),
                p=r.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.999], N).tolist(),
                mp=r.choice([0.0, 0.0, 0.01, 0.3, 1.0], N).tolist())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V", [(1, 1), (9, 2), (40, 7), (33, 64), (40, 65), (64, 1000),
                                 (40, 4097), (3, 8191), (24, 32000), (1, 128256), (16, 128256),
                                 (5, 131072), (6, 256003), (3, 300001)])
def test_mixed(N, V, dtype):
    run(normal(N, V, dtype, N + V), **params(N, V))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 3, 300])
def test_rows_of_a_batch(N, dtype):
    """One row, a few and many: whatever splits the work."""
    run(normal(N, 20011, dtype, N), **params(N, 7 + N))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [100, 32000, 140000])
def test_all_equal(V, dtype):
    """Every logit the same: only the index order decides, at every border."""
    us = [0.0, 0.25, 0.5, 0.999, 1 - 2.0 ** -24, 0.1]
    z = torch.full((len(us), V), 2.5, dtype=DT[dtype], device="cuda")
    run(z, us)
    run(z, us, k=[1, 2, 50, V // 2, V - 1, V])
    run(z, us, p=[0.5, 0.25, 0.125, 0.0, 0.75, 0.9])
    run(z, us, k=[64, 2, 50, V // 2, V - 1, V], p=[0.5, 0.25, 0.125, 0.0, 0.75, 0.9])
    run(z, us, T=[0.0, 1e-30, 1e30, 1.0, 5.0, 0.0], mp=[1.0] * 6)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_few_distinct_values(dtype):
    """Ties at every threshold."""
    N, V = 48, 30000
    g = torch.Generator().manual_seed(3)
    z = torch.randint(-3, 4, (N, V), generator=g).to(DT[dtype]).cuda()
    run(z, **params(N, 5))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sigma", [0.0, 1e-6, 0.05, 1.0, 30.0, 1e4])
def test_spreads(sigma, dtype):
    """From flat rows, where the kept sets are large, to rows of one token."""
    run(normal(20, 40000, dtype, 11, sigma), **params(20, 12))
    run(normal(20, 40000, dtype, 13, sigma) + 1000, **params(20, 14))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mask", [-INF, -FMAX, -1e30, -1e4])
def test_masks(mask, dtype):
    z = normal(24, 20000, dtype, 15)
    g = torch.Generator().manual_seed(16)
    z[torch.rand(z.shape, generator=g).cuda() < 0.999] = mask
    z[3] = mask
    z[4, 1:] = mask
    z[5, :-1] = mask
    run(z, **params(24, 17))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_special_values(dtype):
    N, V = 12, 5000
    z = normal(N, V, dtype, 18)
    z[0, 77] = NAN
    z[1] = -INF
    z[2, [5, 900, 4999]] = INF
    z[3, [5, 900, 4999]] = INF
    z[4] = FMAX
    z[5, ::2], z[5, 1::2] = 0.0, -0.0
    z[6] = NAN
    z[7, 1] = INF
    z[8] = INF
    u = [0.3, 0.3, 0.5, 0.9, 0.7, 0.6, 0.2, 0.99, 0.999, 0.1, 0.2, 0.3]
    run(z, u)
    run(z, u, k=[2] * N)
    run(z, u, p=[0.6] * N)
    run(z, u, T=[0.0] * N)


def test_bad_parameters_give_no_token():
    N = 14
    z = normal(N, 300, "fp32", 19)
    u = [0.5, 1.0, -0.1, NAN, INF] + [0.5] * 9
    T = [-1.0, 1, 1, 1, 1, NAN, INF, -0.0, 1, 1, 1, 1, 1, 1]
    p = [1] * 8 + [NAN, -1.0, 2.0, 1, 1, 1]
    mp = [0] * 11 + [NAN, -1.0, 7.0]
    tok = run(z, u, T=T, p=p, mp=mp)
    assert (tok.cpu() < 0).tolist() == [True] * 7 + [False, True, False, False, True, False,
                                                     False]


def test_views_and_strides():
    """Transposed tokens, rows at odd offsets, one row read many times."""
    z = normal(30, 1003, "bf16", 20).view(5, 6, 1003)
    u = np.random.default_rng(21).random(30, dtype=np.float32).reshape(6, 5)
    zt = z.transpose(0, 1)
    tok = vce.ce_sample(zt, t32(u))
    assert tok.shape == (6, 5)
    flat = vce.ce_sample(zt.reshape(30, 1003).contiguous(), t32(u.reshape(-1)))
    assert torch.equal(tok.reshape(-1), flat)
    for dtype in ("bf16", "fp32"):
        big = normal(8, 4000, dtype, 22)
        for a, b in ((0, 3999), (1, 3001), (3, 7), (5, 3990), (7, 8)):
            run(big[:, a:b], **params(8, a))
        run(big[:1].expand(6, 4000), [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], k=[50] * 6)


def test_outputs_and_neighbours():
    z = normal(4, 500, "fp32", 23)
    u = t32([0.1, 0.5, 0.7, 0.9])
    tok = torch.full((6,), 99, dtype=torch.int64, device="cuda")
    lp = torch.full((6,), 99.0, device="cuda")
    got = vce.ce_sample(z, u, with_logprob=True, out=(tok[1:5], lp[1:5]))
    ref = vce.ce_sample(z, u, with_logprob=True)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert tok[0] == 99 and tok[5] == 99 and lp[0] == 99 and lp[5] == 99
    assert vce.ce_sample(torch.empty((0, 500), device="cuda"), torch.empty(0, device="cuda")
                         ).shape == (0,)


def test_streams_and_graph():
    N, V = 6, 60000
    z = normal(N, V, "bf16", 24)
    k = torch.full((N,), 50, dtype=torch.int32, device="cuda")
    p = torch.full((N,), 0.9, device="cuda")
    u = torch.rand(N, device="cuda")
    ref = vce.ce_sample(z, u, None, k, p, with_logprob=True)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [vce.ce_sample(z, u, None, k, p, with_logprob=True, stream=s)
            for _ in range(4) for s in (a, b)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])
    ws = vce.ce_sample_workspace(N, V)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tok, lp = vce.ce_sample(z, u, None, k, p, with_logprob=True, workspace=ws)
        plain = vce.ce_sample(z, u, workspace=ws)
    for r in range(4):
        z.copy_(normal(N, V, "bf16", 25 + r))
        u.copy_(torch.rand(N, device="cuda"))
        ws.fill_(255)
        g.replay()
        e = vce.ce_sample(z, u, None, k, p, with_logprob=True)
        ep = vce.ce_sample(z, u)
        torch.cuda.synchronize()
        assert torch.equal(tok, e[0]) and torch.equal(lp, e[1]) and torch.equal(plain, ep)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [5000, 50000, 200003])
def test_large_top_k(V, dtype):
    """Top-k beyond what a row's candidates have room for, alone and with the rest; with k at
    and beside the number of tokens above a mask."""
    N, live = 24, V // 3
    z = normal(N, V, dtype, 21)
    z[12:, live:] = -INF
    ks = [1024, 1025, 4096, 4097, 4100, V // 2, V - 1, V, live - 1, live, live + 1, V // 5]
    u = np.random.default_rng(22).random(N, dtype=np.float32).tolist()
    run(z, u, k=ks * 2)
    run(z, u, k=ks * 2, T=[3.0, 0.2] * 12, mp=[0.0, 1e-3, 0.3] * 8)
    run(z, u, k=ks * 2, p=[0.999, 0.5] * 12)
    run(torch.round(z), u, k=ks * 2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [129, 1000, 4095, 4096])
def test_short_rows(V, dtype):
    """Rows that are served whole, with every filter alone and together."""
    N = 40
    z = normal(N, V, dtype, V)
    z[:10] = torch.round(z[:10])
    z[10:15, ::2] = -INF
    g = params(N, V + 1)
    run(z, g["u"])
    run(z, g["u"], T=g["T"])
    run(z, g["u"], k=[1, 7, 8, 30, 100, V // 2, V - 1, V] * 5)
    run(z, g["u"], p=g["p"])
    run(z, g["u"], mp=[1e-6, 0.01, 0.5, 1.0] * 10)
    run(z, **g)


@pytest.mark.parametrize("N,V", [(256, 5000), (257, 5000), (32, 60000), (33, 60000)])
def test_few_and_many_segments(N, V):
    """At and past the number of row segments up to which a row's workgroups join."""
    z = normal(N, V, "bf16", N)
    g = params(N, N)
    run(z, **g)
    ws = vce.ce_sample_workspace(N, V)
    ws.fill_(255)
    args = [t32(g["T"]), torch.tensor(g["k"], dtype=torch.int32, device="cuda"), t32(g["p"]),
            t32(g["mp"])]
    first = vce.ce_sample(z, t32(g["u"]), *args, with_logprob=True, workspace=ws)
    for _ in range(3):  # what a call leaves in the workspace means nothing to the next
        again = vce.ce_sample(z, t32(g["u"]), *args, with_logprob=True, workspace=ws)
        assert torch.equal(first[0], again[0])
        assert torch.equal(first[1].nan_to_num(7.0), again[1].nan_to_num(7.0))
