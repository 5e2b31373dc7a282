"""The beam search step against the FP64 reference (parents and tokens equal), and the
reordering of states against indexing."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, U, f64
from oracle import beam

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def logits(B, K, V, dtype, seed, sigma=3.0, pad=0, skew=0):
    """(B, K, V) with rows `pad` tokens apart, `skew` elements past an allocation."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((skew + B * K * (V + pad),), NAN, dtype=DT[dtype], device="cuda")
    z = buf[skew:].view(B, K, V + pad)[:, :, :V]
    z.copy_(torch.randn((B, K, V), generator=g) * sigma)
    s = -20 * torch.rand((B, K), generator=g)
    return z, s.cuda()


def check(z, s, n_out=None, ended=None, end_token=0, got=None):
    B, K, V = z.shape
    n = n_out or K
    if got is None:
        got = vce.beam_step(z, s, n_out, ended=ended, end_token=end_token)
    score, parent, token = (t.cpu().numpy() for t in got)
    zz, ss = f64(z), f64(s)
    for b in range(B):
        v, p, t = beam.step(zz[b], ss[b], n, None if ended is None else ended[b].tolist(),
                            end_token)
        assert parent[b].tolist() == p.tolist() and token[b].tolist() == t.tolist(), b
        # FP64 until the last rounding (lse to 1e-11 at most)
        fin = np.isfinite(v)
        assert (score[b][~fin] == v[~fin]).all()
        assert (np.abs(score[b][fin] - v[fin]) <= U * np.abs(v[fin]) + 2e-11).all()
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,K,V,n_out,pad,skew", [
    (1, 1, 1, 1, 0, 0), (1, 1, 5, 8, 0, 0), (2, 3, 2, 6, 1, 1), (1, 4, 32000, 4, 0, 0),
    (3, 5, 8191, 10, 0, 0), (2, 2, 8192, 4, 0, 0), (2, 2, 8193, 4, 7, 3), (16, 8, 1000, 8, 0, 0),
    (2, 8, 50257, 16, 0, 1), (1, 16, 128256, 32, 0, 0), (5, 5, 32003, 10, 5, 2),
    (1, 1, 256003, 64, 0, 0), (1, 128, 3001, 256, 0, 0), (2, 33, 9000, 66, 0, 0),
    (1, 3, 100000, 256, 0, 0), (300, 2, 70, 4, 0, 0), (1, 64, 40000, 128, 0, 0)])
def test_step(B, K, V, n_out, pad, skew, dtype):
    z, s = logits(B, K, V, dtype, B * K + V, pad=pad, skew=skew)
    check(z, s, n_out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sigma", [0.0, 1e-4, 0.05, 30.0])
@pytest.mark.parametrize("V", [700, 20001])
def test_flat_and_steep(V, sigma, dtype):
    """Rows that tie everywhere (more candidates than the lists hold), nearly, or hardly."""
    z, s = logits(2, 6, V, dtype, 3, sigma)
    check(z, s, 12)
    s.fill_(-1.0)
    check(z, s, 6)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_equal_beams(dtype):
    """Beams with equal rows and scores tie exactly, at any alignment: the lower beam first."""
    z, s = logits(2, 4, 12345, dtype, 9, pad=3, skew=1)
    z[:, 1:] = z[:, :1].clone()
    s[:, 1:] = s[:, :1].clone()
    _, parent, token = check(z, s, 8)
    assert parent[:, :4].tolist() == [[0, 1, 2, 3]] * 2
    assert bool((token[:, :4] == token[:, :1]).all())


@pytest.mark.parametrize("V", [40, 9000, 30000])
def test_masks(V):
    z, s = logits(9, 4, V, "fp32", 4)
    z[0, 1] = -INF                       # nothing left of a beam
    z[1] = -INF                          # of a request
    z[2, 0, V // 2] = NAN
    z[3, 3, 7] = INF
    z[4, :, 3:] = -INF                   # fewer candidates than asked for
    z[5, :, : V - 1] = -3.4e38           # a finite mask, one token above it
    z[6, 2] = torch.where(torch.rand(V, device="cuda") < 0.9, -INF, z[6, 2])
    z[7, 0, 1:] = -INF                   # one token: certain
    z[8, :, 8:] = -INF
    check(z, s, 16)
    s[0, 0], s[2, 1], s[3, 2], s[6, 0] = -INF, NAN, INF, -INF
    check(z, s, 16)
    s[8, 1:] = -INF                      # a first step: one beam
    check(z, s, 4)
    s.fill_(-INF)
    score, parent, token = check(z, s, 4)
    assert bool((parent == -1).all()) and bool((token == -1).all()) and bool((score == -INF).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,end", [(50, 49), (20000, 3)])
def test_ended(V, end, dtype):
    z, s = logits(6, 5, V, dtype, 8)
    ended = torch.zeros((6, 5), dtype=torch.bool, device="cuda")
    ended[0, 2] = ended[1, :] = ended[2, 0] = ended[3, 1] = ended[3, 4] = True
    s[0, 2], s[2, 0], s[3, 1] = -0.5, -200.0, -INF
    z[1] = NAN                           # not read
    z[3, 4] = INF
    s[4, 0] = s[4, 1] = -1.0
    ended[4, :2] = True                  # two that tie
    check(z, s, 10, ended, end)
    check(z, s, None, ended, end)


def test_layouts():
    """Beams before requests, one row read by all, a request's rows far apart."""
    z, s = logits(3, 4, 5001, "bf16", 1)
    check(z.transpose(0, 1).contiguous().transpose(0, 1), s, 8)
    check(z[:1, :1].expand(3, 4, 5001), s, 8)
    far = torch.empty((1 << 31) + 9001, dtype=torch.bfloat16, device="cuda")
    y = far.as_strided((2, 2, 5000), (5000, (1 << 31) - 7000, 1))
    y.copy_(z[:2, :2, :5000])
    check(y, s[:2, :2].contiguous(), 8)


def test_workspace_and_outputs():
    """No byte beyond the workspace or the outputs."""
    for B, K, V in ((1, 1, 10), (3, 5, 9000)):
        z, s = logits(B, K, V, "fp32", 2)
        n = vce.beam_workspace_size(B, K, V)
        buf = torch.full((n + 512,), 170, dtype=torch.uint8, device="cuda")
        outs = [torch.full((B * 4 + 8,), 7, dtype=d, device="cuda")
                for d in (torch.float32, torch.int32, torch.int64)]
        out = [t[:B * 4].view(B, 4) for t in outs]
        check(z, s, 4, got=vce.beam_step(z, s, 4, workspace=buf[:n], out=out))
        assert bool((buf[n:] == 170).all()) and all(bool((t[B * 4:] == 7).all()) for t in outs)


# ---- reordering ------------------------------------------------------------------------

def parents(B, K, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, K, (B, K), generator=g, dtype=torch.int32).cuda()


def want(t, parent):
    B, K = parent.shape
    p = torch.where((parent < 0) | (parent >= K), torch.arange(K, device="cuda"), parent.long())
    return torch.stack([t[b][p[b]] for b in range(B)])


def check_reorder(states, parent):
    ref = [want(t, parent) for t in states]
    vce.beam_reorder(states, parent)
    for i, (t, r) in enumerate(zip(states, ref)):
        assert torch.equal(t, r), i


@pytest.mark.parametrize("B,K", [(1, 1), (2, 3), (5, 8), (3, 9), (2, 32), (2, 33), (1, 128)])
def test_reorder(B, K):
    g = torch.Generator(device="cuda").manual_seed(K)
    r = lambda *s, d=torch.int64: torch.randint(0, 100, s, generator=g, device="cuda").to(d)
    states = [r(B, K, 37), r(B, K), r(B, K, 5003, d=torch.bfloat16), r(B, K, 1, d=torch.uint8),
              r(B, K, 7, 3, d=torch.int8), r(B, K, 4096, d=torch.float32), r(B, K, 0),
              r(B, K, 2, 16, 5, d=torch.float64)]
    check_reorder(states, parents(B, K, 1))
    same = torch.arange(K, dtype=torch.int32, device="cuda").repeat(B, 1)
    check_reorder(states, same)
    check_reorder(states, same.flip(1).contiguous())
    check_reorder(states, torch.zeros_like(same))
    odd = parents(B, K, 2)
    odd[:, 0], odd[0, K - 1] = -1, K  # no such beam: the row stays
    check_reorder(states, odd)
    wide = parents(B, 2 * K, 3) % K
    check_reorder(states, wide[:, :K])


def test_reorder_views():
    """The used part of longer caches, slices of one array, requests behind beams, odd addresses;
    what lies between the pieces stays."""
    B, K = 3, 4
    p = parents(B, K, 5)
    full = torch.randn((B, K, 6, 50, 8), device="cuda")
    keep = full.clone()
    check_reorder([full[:, :, :, :33]], p)
    assert torch.equal(full[:, :, :, 33:], keep[:, :, :, 33:])
    both = torch.randn((B, K, 2, 100), device="cuda")
    check_reorder([both[:, :, 0], both[:, :, 1]], p)
    pair = torch.randn((B, K, 10, 2, 6), device="cuda")
    check_reorder([pair[:, :, :, 0], pair[:, :, :, 1]], p)
    check_reorder([torch.randn((K, B, 77), device="cuda").transpose(0, 1)], p)
    raw = torch.randint(0, 255, (B * K * 101 + 3,), dtype=torch.uint8, device="cuda")
    rim = raw.clone()
    view = raw[3:].view(B, K, 101)[:, :, :67]
    check_reorder([view], p)
    raw[3:].view(B, K, 101)[:, :, :67] = rim[3:].view(B, K, 101)[:, :, :67]
    assert torch.equal(raw, rim)


def test_reorder_many_and_large():
    """More states than a launch's table; a state past 2^32 bytes."""
    p = parents(2, 5, 6)
    check_reorder([torch.randn((2, 5, 10 + i), device="cuda") for i in range(100)], p)
    big = torch.zeros((1, 2, (1 << 31) + 21), dtype=torch.uint8, device="cuda")
    big[0, 0, ::4097], big[0, 1, ::4099] = 3, 5
    big[0, 0, -1], big[0, 1, -1] = 7, 9
    vce.beam_reorder(big, torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    assert big[0, 1, -1] == 7 and big[0, 0, -1] == 9
    a, b = torch.zeros_like(big[0, 0]), torch.zeros_like(big[0, 0])
    a[::4097], b[::4099] = 3, 5
    a[-1], b[-1] = 7, 9
    assert torch.equal(big[0, 0], b) and torch.equal(big[0, 1], a)


# ---- a search ------------------------------------------------------------------------------

def step(z, s, hist, cache, ended, at, ws=None, out=None, stream=None):
    score, parent, token = vce.beam_step(z, s, ended=ended, end_token=1, workspace=ws, out=out,
                                         stream=stream)
    vce.beam_reorder([hist, cache], parent, stream=stream)
    return score, parent, token


def test_search_captured():
    """A step with its reordering captured once and replayed over new logits, against eager runs."""
    B, K, V = 3, 4, 9001
    z, s = logits(B, K, V, "bf16", 1)
    ended = torch.zeros((B, K), dtype=torch.bool, device="cuda")
    hist = torch.zeros((B, K, 9), dtype=torch.int64, device="cuda")
    cache = torch.randn((B, K, 100), device="cuda")
    h2, c2 = hist.clone(), cache.clone()
    ws = vce.beam_workspace(B, K, V)
    out = vce.beam_step(z, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(z, s, hist, cache, ended, 0, ws, out)
    for i in range(4):
        z.copy_(logits(B, K, V, "bf16", 10 + i)[0])
        ended.copy_(torch.rand((B, K), device="cuda") < 0.2)
        graph.replay()
        score, parent, token = check(z, s, None, ended, 1,
                                     got=step(z, s, h2, c2, ended, i))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (score, parent, token)))
        assert torch.equal(hist, h2) and torch.equal(cache, c2)
        for h in (hist, h2):
            h[:, :, i] = token
        s.copy_(score)


def test_two_streams():
    cases = [logits(2, 8, 30000, "bf16", 1), logits(4, 3, 5000, "fp32", 2)]
    want = [vce.beam_step(z, s) for z, s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [vce.beam_step(z, s, stream=t) for t, (z, s) in zip(streams, cases)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
