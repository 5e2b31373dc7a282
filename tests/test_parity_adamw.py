"""The optimizer step and the gradients' norm against FP64, the 8-bit states bit by bit
against FP32 arithmetic rounded operation by operation."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, HALF, TINY, U, assert_within, f64
from oracle import head, step as ref

pytestmark = pytest.mark.gpu

B1, B2, EPS, WD, LR = 0.9, 0.999, 1e-8, 0.01, 1e-3


def make(sizes, pd, gd, seed, bits=32, master=False, skew=0):
    """Parameters and gradients (at `skew` elements past an allocation) and a state in midway."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=g)

    def place(t, dtype):
        buf = torch.full((t.numel() + skew + 8,), 7.0, dtype=DT[dtype], device="cuda")
        buf[skew:skew + t.numel()] = t.to(DT[dtype])
        return buf[skew:skew + t.numel()]
    params = [place(rnd(n) * 0.02, pd) for n in sizes]
    grads = [place(rnd(n) * 1e-3 * torch.exp(2 * rnd(n)), gd) for n in sizes]
    st = vce.adamw_state(params, bits, master)
    for n, o in zip(st.sizes, st.offsets):
        if n == 0:
            continue
        m, r = rnd(n) * 3e-4 * torch.exp(rnd(n)), 1e-3 * torch.exp(rnd(n))
        if bits == 32:
            st.m[o:o + n], st.v[o:o + n] = m.cuda(), (r * r).cuda()
        else:
            for t, q, s in ((m, st.m, st.m_scales), (r, st.v, st.v_scales)):
                pad = torch.zeros((n + 31) // 32 * 32)
                pad[:n] = t
                a, b = vce.mx_quantize(pad.view(1, -1).cuda(), "e4m3")
                q[o:o + a.numel()], s[o // 32:o // 32 + b.numel()] = a.view(-1), b.view(-1)
    return params, grads, st


def moments(st):
    """(m, v) as FP64 over the flat places."""
    if st.bits == 32:
        return f64(st.m), f64(st.v)
    m, r = (head.dequantize(q.cpu().numpy().reshape(1, -1), s.cpu().numpy().reshape(1, -1),
                            "e4m3").reshape(-1)
            for q, s in ((st.m, st.m_scales), (st.v, st.v_scales)))
    return m, r * r


def check(params, grads, st, call, scale=1.0, step=3, lr=LR, betas=(B1, B2), eps=EPS, wd=WD,
          seed=0):
    """`call()` runs the step; parameters, masters and states against their references."""
    b1, b2 = betas
    old = [f64(p) for p in params] if st.master is None else \
        [f64(st.master[o:o + n]) for n, o in zip(st.sizes, st.offsets)]
    m0, v0 = moments(st)
    gs = [None if g is None else f64(g) for g in grads]
    before = {k: getattr(st, k).clone() for k in ("m", "v", "m_scales", "v_scales")
              if getattr(st, k) is not None}
    kept = [p.clone() for p in params]
    call()
    for i, (n, o) in enumerate(zip(st.sizes, st.offsets)):
        at, end = slice(o, o + n), o + (n + 127) // 128 * 128
        if gs[i] is None or n == 0:
            assert torch.equal(params[i], kept[i])
            assert torch.equal(st.m[o:end], before["m"][o:end])
            continue
        g, m, v = gs[i] * scale, m0[at], v0[at]
        p1, m1, v1 = ref.adamw(old[i], g, m, v, lr, step, b1, b2, eps, wd)
        # m: the constants, products, the scaled gradient and the sum, each one rounding of a
        # term of size S; v: the same with the square; both terms positive
        S = b1 * np.abs(m) + (1 - b1) * np.abs(g)
        bm, bv = 5 * U * S + TINY, 8 * U * v1 + TINY
        if st.bits == 32:
            assert_within(f64(st.m[at]), m1, bm, f"m {i}")
            assert_within(f64(st.v[at]), v1, bv, f"v {i}")
        else:
            a, b = ref.moments32(gs[i].astype(np.float32), scale, m, v, b1, b2)
            r = ref.random_bits(np.arange(o, end), seed, step)
            pad = np.zeros(end - o, np.float32)
            for x, q, s, r16, keep in ((a, st.m, st.m_scales, r & np.uint64(65535), False),
                                       (np.sqrt(b), st.v, st.v_scales, r >> np.uint64(16), True)):
                pad[:n] = x
                code, sc = ref.round_random(pad, r16, keep)
                used = (n + 31) // 32
                assert np.array_equal(q[o:end].cpu().numpy(), code), f"codes {i}"
                assert np.array_equal(s[o // 32:o // 32 + used].cpu().numpy(), sc[:used])
        # p: decay (constant, product, difference: 3 u of p); the step: m's error above,
        # root 4.5 u with v's, the reciprocal 1 ulp = 2 u, eps and the factors 5 u, products 2 u
        bc1, bc2 = 1 - b1 ** step, 1 - b2 ** step
        # v may also lie 2^-148 off: below the normal range its old value's square, g'^2, the two
        # products and their sum are each rounded by 2^-150 at most (the sum exactly).  The root of
        # an interval around v then bounds the step.
        d = np.sqrt(v1 / bc2) + eps
        lo = np.sqrt(np.maximum(v1 - 2.0 ** -148, 0) / bc2) + eps
        hi = np.sqrt((v1 + 2.0 ** -148) / bc2) + eps
        with np.errstate(all="ignore"):
            size = lr / bc1 * S / d
            spread = np.where(lo > 0, lr / bc1 * np.abs(m1) * (1 / lo - 1 / hi), 0)
        bp = 3 * U * np.abs(old[i]) + 20 * U * (size + spread) + spread + TINY
        if st.master is not None:
            assert_within(f64(st.master[at]), p1, bp + U * np.abs(p1), f"master {i}")
            assert bool((st.master[o + n:end] == 0).all())
        h = HALF[params[i].dtype]
        assert_within(f64(params[i]), p1, bp + h * (np.abs(p1) + bp), f"p {i}")
        assert bool((st.m[o + n:end] == 0).all()) and bool((st.v[o + n:end] == 0).all())


SIZES = [1, 7, 8, 31, 32, 33, 127, 128, 129, 1000, 4095, 4096, 4097, 12289, 0, 5]


@pytest.mark.parametrize("skew", [0, 1, 4])
@pytest.mark.parametrize("pd,gd", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"),
                                   ("fp32", "bf16")])
@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_step(bits, master, pd, gd, skew):
    P, G, st = make(SIZES, pd, gd, 11, bits, master, skew)
    check(P, G, st, lambda: vce.adamw_step(P, G, st, LR, 3, weight_decay=WD))
    for t in P + G:  # and nothing beside the tensors
        n = t.numel() if t.numel() else 1
        rim = torch.as_strided(t, (8,), (1,), t.storage_offset() + t.numel())
        assert bool((rim == 7.0).all()), n


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("betas,eps,wd,step,lr", [
    ((0.0, 0.0), 1e-8, 0.0, 1, 1e-2), ((0.9, 0.999), 0.1, 0.5, 1, 1.0),
    ((0.95, 0.98), 0.0, 0.0, 1000000, 0.0), ((0.5, 0.9999), 1e-12, 0.1, 1 << 40, 3e-4)])
def test_parameters(bits, betas, eps, wd, step, lr):
    P, G, st = make([300, 5000], "fp32", "fp32", 5, bits)
    check(P, G, st, lambda: vce.adamw_step(P, G, st, lr, step, betas=betas, eps=eps,
                                           weight_decay=wd, seed=1 << 40 | 9),
          step=step, lr=lr, betas=betas, eps=eps, wd=wd, seed=1 << 40 | 9)


@pytest.mark.parametrize("bits", [8, 32])
def test_first_step_from_zero(bits):
    g = torch.Generator().manual_seed(1)
    P = [(torch.randn(3000, generator=g)).cuda()]
    G = [(torch.randn(3000, generator=g) * 1e-2).cuda()]
    G[0][:700] = 0  # rows without a gradient: nothing but the decay
    st = vce.adamw_state(P, bits)
    check(P, G, st, lambda: vce.adamw_step(P, G, st, LR, 1, weight_decay=WD), step=1)


@pytest.mark.parametrize("scale", [1e-37, 1e-30, 1e-21, 1e-12, 1e6, 1e17])
@pytest.mark.parametrize("bits", [8, 32])
def test_small_and_large(bits, scale):
    """Gradients far from one, down to where their squares leave FP32's normal range."""
    P, G, st = make([700], "fp32", "fp32", 6, bits)
    st.m.zero_(), st.v.zero_()
    G[0] *= scale / 1e-3
    G[0][64:128] *= 1e-5
    if 0.1 * scale < 2.0 ** -126:  # an eps below FP32's normal range is refused
        with pytest.raises(vce.VceError, match="VCE_EINVAL"):
            vce.adamw_step(P, G, st, LR, 1, eps=0.1 * scale)
        return
    for step in (1, 2):
        check(P, G, st, lambda: vce.adamw_step(P, G, st, LR, step, eps=0.1 * scale,
                                               weight_decay=WD), step=step, eps=0.1 * scale)


def test_many_tensors_shapes_and_none():
    """More than a launch's table, shapes of two dimensions, absent gradients."""
    r = np.random.default_rng(3)
    sizes = [int(t) for t in r.integers(1, 3000, 150)]
    P, G, st = make(sizes, "bf16", "fp32", 8, 8)
    G = [None if i % 7 == 3 else t for i, t in enumerate(G)]
    check(P, G, st, lambda: vce.adamw_step(P, G, st, LR, 3, weight_decay=WD))
    W = torch.randn((33, 70), device="cuda")
    D, s2 = torch.randn((33, 70), device="cuda"), vce.adamw_state([W])
    check([W.view(-1)], [D.view(-1)], s2,
          lambda: vce.adamw_step([W], [D], s2, LR, 1, weight_decay=WD), step=1)
    vce.adamw_step([W], [None], s2, LR, 2)


@pytest.mark.parametrize("bits", [8, 32])
def test_scale_and_device_scalars(bits):
    P, G, st = make([900, 4100], "fp32", "bf16", 21, bits)
    sc = torch.tensor(0.37, device="cuda")
    lr, step = torch.tensor(2e-3, device="cuda"), torch.tensor([17], device="cuda")
    check(P, G, st, lambda: vce.adamw_step(P, G, st, lr, step, weight_decay=WD, grad_scale=sc),
          scale=float(sc), step=17, lr=float(lr))
    for bad in (float("nan"), float("inf"), -float("inf")):
        sc.fill_(bad)
        kept = [t.clone() for t in P + [st.m, st.v]]
        vce.adamw_step(P, G, st, lr, step, grad_scale=sc)
        assert all(torch.equal(a, b) for a, b in zip(kept, P + [st.m, st.v]))


def test_captured():
    """A captured step follows its device scalars and gradients; norm and step in one graph."""
    P, G, st = make([5000, 33], "bf16", "bf16", 2, 8)
    Q = [p.clone() for p in P]
    lr, step = torch.tensor(1e-3, device="cuda"), torch.tensor(4, device="cuda")
    out = (torch.empty((), device="cuda"), torch.empty((), device="cuda"))
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    eager = vce.adamw_state(Q, 8)

    def both(params, state):
        vce.grad_norm(G, 0.5, out=out, workspace=ws)
        vce.adamw_step(params, G, state, lr, step, grad_scale=out[1], seed=77)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(P, st)
    for a in ("m", "v", "m_scales", "v_scales"):
        getattr(eager, a).copy_(getattr(st, a))
    for i in range(4):
        for t in G:
            t.copy_(torch.randn(t.shape, device="cuda") * 10.0 ** -i)
        lr.fill_(1e-3 * (i + 1))
        step.fill_(4 + i)
        graph.replay()
        got = out[0].item(), out[1].item()
        both(Q, eager)
        torch.cuda.synchronize()
        assert got == (out[0].item(), out[1].item())
        for a, b in zip(P + [st.m, st.v, st.m_scales, st.v_scales],
                        Q + [eager.m, eager.v, eager.m_scales, eager.v_scales]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("bits", [8, 32])
def test_not_finite(bits):
    """A NaN or an infinity stays where it is: its element, or its block of 32 in 8 bits."""
    P, G, st = make([200], "fp32", "fp32", 4, bits)
    clean = [t.clone() for t in (P[0], st.m, st.v)]
    scales = [None if s is None else s.clone() for s in (st.m_scales, st.v_scales)]
    vce.adamw_step(P, G, st, LR, 3)
    want = [t.clone() for t in (P[0], st.m, st.v)]
    for t, c in zip((P[0], st.m, st.v), clean):
        t.copy_(c)
    if bits == 8:
        st.m_scales.copy_(scales[0])
        st.v_scales.copy_(scales[1])
    G[0][40], G[0][70] = float("nan"), float("inf")
    vce.adamw_step(P, G, st, LR, 3)
    ok = torch.ones(200, dtype=torch.bool)
    ok[[40, 70]] = False
    assert torch.equal(P[0].cpu()[ok], want[0].cpu()[ok])
    assert bool(P[0][40].isnan())
    m, v = moments(st)
    if bits == 32:
        assert np.isnan(m[40]) and np.isinf(m[70]) and np.isinf(v[70])
        assert torch.equal(st.m[:200].cpu()[ok], want[1][:200].cpu()[ok])
    else:
        assert np.isnan(m[32:96]).all() and np.isnan(v[32:96]).all()
        ok = torch.ones(256, dtype=torch.bool)
        ok[32:96] = False
        assert torch.equal(st.m.cpu()[ok], want[1].cpu()[ok])
        assert torch.equal(st.v.cpu()[ok], want[2].cpu()[ok])


def test_rounding_keeps_the_mean():
    """The mean of 2^16 values rounded at random lies within six standard errors of the value:
    a step h of the grid at part t has variance h^2 t (1 - t), and 16 bits add at most h 2^-16."""
    n = 1 << 16
    for part in (0.002, 0.3, 0.75):
        P, G = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
        x = 2.0 ** -10 * (1 + part / 8)  # between two codes, its block's scale a power of two
        G[0].fill_(x)
        st = vce.adamw_state(P, 8)
        vce.adamw_step(P, G, st, 0.0, 9, betas=(0.0, 0.0), seed=5)
        m, v = moments(st)
        h = 2.0 ** -13
        bound = h * (6 * np.sqrt(part * (1 - part) / n) + 2.0 ** -16) + 4 * U * x
        assert abs(m.mean() - x) <= bound and abs(np.sqrt(v).mean() - x) <= bound, part
        assert len(np.unique(m)) == 2
        # neighbouring places and steps are rounded apart from one another: so many ups in
        # common as chance gives, within six standard deviations
        up = m > x
        vce.adamw_step(P, G, st, 0.0, 10, betas=(0.0, 0.0), seed=5)
        again = moments(st)[0] > x
        for a, b in ((up[:-1], up[1:]), (up, again), (up, np.sqrt(v) > x)):
            p = part * part
            assert abs((a & b).mean() - p) <= 6 * np.sqrt(p / n) + 4 * 2.0 ** -16, part


@pytest.mark.parametrize("gd", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 3], [16384], [16385, 7, 40000],
                                   [3] * 70 + [20001]])
def test_norm(sizes, gd):
    _, G, _ = make([max(1, n) for n in sizes], "fp32", gd, 6, skew=1)
    G = [g[:n] for g, n in zip(G, sizes)]
    total = np.sqrt(sum((f64(g) ** 2).sum() for g in G))
    for most in (float("inf"), float(total) * 2, float(total) * 0.3):
        norm, scale = vce.grad_norm(G, most)
        # FP64 until the last rounding
        assert abs(norm.item() - total) <= 2 * U * total
        want = min(1.0, most / total)
        assert abs(scale.item() - want) <= 2 * U * want
        again = vce.grad_norm(G + [None], most)
        assert torch.equal(norm, again[0]) and torch.equal(scale, again[1])


def test_norm_edges():
    G = [torch.zeros(100, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.bfloat16)]
    norm, scale = vce.grad_norm(G, 1.0)
    assert norm.item() == 0.0 and scale.item() == 1.0
    G[0][3] = 3e38  # its square passes FP32, not FP64
    norm, scale = vce.grad_norm(G, 1.0)
    big = float(G[0][3])
    assert abs(norm.item() - big) <= U * big and abs(scale.item() * big - 1) <= 2 * U
    for bad in (float("inf"), float("nan")):
        G[1][0] = bad
        norm, scale = vce.grad_norm(G, 1.0)
        assert not np.isfinite(norm.item()) and np.isnan(scale.item())


def test_two_streams():
    a, b = make([50000, 7], "bf16", "bf16", 1, 8), make([33, 70000], "fp32", "fp32", 2)
    want = []
    for P, G, st in (a, b):
        P2, s2 = [p.clone() for p in P], vce.adamw_state(P, st.bits)
        for k in ("m", "v", "m_scales", "v_scales"):
            if getattr(st, k) is not None:
                getattr(s2, k).copy_(getattr(st, k))
        for i in range(3):
            vce.adamw_step(P2, G, s2, LR, i + 1, grad_scale=vce.grad_norm(G, 0.1)[1])
        want.append(P2 + [s2.m, s2.v])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(3):
        for s, (P, G, st) in zip(streams, (a, b)):
            sc = vce.grad_norm(G, 0.1, stream=s)[1]
            vce.adamw_step(P, G, st, LR, i + 1, grad_scale=sc, stream=s)
    torch.cuda.synchronize()
    for w, (P, G, st) in zip(want, (a, b)):
        assert all(torch.equal(x, y) for x, y in zip(w, P + [st.m, st.v]))


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("lr,t", [(float("nan"), 1), (float("inf"), 1), (-1e-3, 1), (1e-3, 0), (1e-3, -(1 << 40))])
def test_numbers_on_the_device_that_are_none(lr, t, bits):
    """A rate or a step on the device that the host would refuse: nothing changes."""
    p, g = torch.randn(300, device="cuda"), torch.randn(300, device="cuda")
    st = vce.adamw_state([p], bits)
    vce.adamw_step([p], [g], st, 1e-3, 1)
    held = [x.clone() for x in (p, st.m, st.v)]
    lr_t = torch.tensor([lr], device="cuda")
    t_t = torch.tensor([t], dtype=torch.int64, device="cuda")
    vce.adamw_step([p], [g], st, lr_t, t_t)
    assert all(torch.equal(x, y) for x, y in zip(held, (p, st.m, st.v)))
    vce.adamw_step([p], [g], st, lr_t.fill_(1e-3), t_t.fill_(2))
    assert not torch.equal(held[0], p)
