"""The operators around the head run together, as a server and as a trainer run
them: norm into 8 bits, the product over a microscaled classifier, the draw; and
norm, fused linear cross-entropy and its gradient, the norm's gradient.  Each
stage against its FP64 reference on the stage's own input, then the whole."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import HALF, TINY, U, assert_within, f64, rand
from oracle import head
from vce_testutil import LINEAR_FROB_RTOL, rel_frobenius

pytestmark = pytest.mark.gpu


def serve(x, res, g, w, ws, w_fmt, u, T, k, p, mp, stream=None, buf=None):
    """(q, scales, rstd, h, logits, token, logprob); buf: the same to write into, and a workspace."""
    b = buf or {}
    q, s, rstd, h = vce.rms_forward_mx8(x, g, res, 1e-6, weight_offset=1.0, stream=stream,
                                        out=b.get("norm"))
    z = vce.mx_logits(q, s, w, ws, w_fmt=w_fmt, out=b.get("z"), stream=stream)
    tok, lp = vce.ce_sample(z, u, T, k, p, mp, with_logprob=True, workspace=b.get("work"),
                            out=b.get("draw"), stream=stream)
    return q, s, rstd, h, z, tok, lp


def inputs(M, H, V, w_fmt, seed):
    x, res = rand((M, H), "bf16", seed), rand((M, H), "bf16", seed + 1)
    g = rand((H,), "bf16", seed + 2, 0.1)
    W = rand((V, H), "bf16", seed + 3, 4.0 * H ** -0.5)
    w, ws = vce.mx_quantize(W, w_fmt)
    r = np.random.default_rng(seed)
    t = lambda a, d: torch.tensor(np.asarray(a), dtype=d, device="cuda")
    return (x, res, g, w, ws, w_fmt, t(r.random(M, dtype=np.float32), torch.float32),
            t(r.choice([0.0, 0.7, 1.0], M), torch.float32),
            t(r.choice([0, 1, 20], M), torch.int32), t(r.choice([0.9, 1.0], M), torch.float32),
            t(r.choice([0.0, 0.05], M), torch.float32))


def check_draw(z, a, tok, lp):
    zz, V = f64(z), z.shape[1]
    u, T, k, p, mp = (v.tolist() for v in a[6:])
    ref = [head.sample(zz[i], u[i], T[i], k[i], p[i], mp[i]) for i in range(len(u))]
    assert tok.tolist() == [t for t, _ in ref]
    rl = np.array([l for _, l in ref])
    assert_within(f64(lp), rl, U * np.abs(rl) + V * 2.0 ** -45 + 1e-15, "logprob")


@pytest.mark.parametrize("w_fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,H,V", [(1, 64, 70), (1, 4096, 5000), (7, 512, 32000), (16, 2304, 1001),
                                   (65, 96, 4099), (130, 1024, 300)])
def test_serving(M, H, V, w_fmt):
    a = inputs(M, H, V, w_fmt, M + H)
    x, res, g, w, ws = a[:5]
    q, s, rstd, h, z, tok, lp = serve(*a)
    y, rr, rh = head.rms_forward(f64(x), f64(g), f64(res), 1e-6, 1.0)
    assert_within(f64(h), rh, (HALF[h.dtype] + U) * np.abs(rh) + TINY, "h")
    assert_within(f64(rstd), rr, 64 * U * rr, "rstd")
    sb = s.cpu().numpy()
    dq = head.dequantize(q.cpu().numpy(), sb, "e4m3")
    # y: half a step of the 8 bits at its scale (2^-4 of the value, and below 2^-6 of the
    # scale's unit half of 2^-9), and the norm's own 64 u, also across a step
    unit = np.repeat(2.0 ** (sb.astype(np.float64) - 127), 32, axis=1)
    ybound = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * unit + 2 * 64 * U * np.abs(y)
    assert_within(dq, y, ybound, "y")
    # the product over what the 8 bits hold (the bound of the product's own tests)
    b = head.dequantize(w.cpu().numpy(), ws.cpu().numpy(), w_fmt)
    ref, S = dq @ b.T, np.abs(dq) @ np.abs(b).T
    pk = np.zeros_like(ref)
    for i in range(0, H, 8):  # at most the group's largest product, per group of eight
        pk += np.max(np.abs(dq[:, i:i + 8]), axis=1)[:, None] * \
            np.max(np.abs(b[:, i:i + 8]), axis=1)[None, :]
    own = (HALF[z.dtype] + U) * np.abs(ref) + H * U * S + 2.0 ** -10 * pk
    assert_within(f64(z), ref, own, "logits")
    # and the whole: the 8 bits' rounding spread over the row
    assert_within(f64(z), y @ b.T, own + ybound @ np.abs(b).T, "logits of the whole")
    check_draw(z, a, tok, lp)


@pytest.mark.parametrize("M,H,V", [(1, 512, 5000), (40, 256, 4500)])
def test_serving_graph(M, H, V):
    """Captured with one set of buffers, replayed on changing inputs between eager runs."""
    a = inputs(M, H, V, "e2m1", 5)
    e = lambda *s, d=torch.uint8: torch.empty(s, dtype=d, device="cuda")
    # rows of the logits padded to 16 bytes, as a decode loop keeps them
    zbuf = e(M, (V + 15) // 8 * 8, d=torch.bfloat16)
    zbuf.fill_(7)
    buf = dict(norm=(e(M, H), e(M, H // 32), e(M, d=torch.float32), e(M, H, d=torch.bfloat16)),
               z=zbuf[:, :V], draw=(e(M, d=torch.int64), e(M, d=torch.float32)),
               work=vce.ce_sample_workspace(M, V))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    serve(*a, stream=side, buf=buf)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        serve(*a, buf=buf)
    for i in range(4):
        fresh = inputs(M, H, V, "e2m1", 20 + i)
        for old, new in zip(a, fresh):
            if isinstance(old, torch.Tensor):
                old.copy_(new)
        want = serve(*a)
        graph.replay()
        torch.cuda.synchronize()
        got = buf["norm"] + (buf["z"],) + buf["draw"]
        for n, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), (i, n)
        check_draw(buf["z"], a, *buf["draw"])
    assert bool((zbuf[:, V:] == 7).all())


def test_serving_two_streams():
    """Two chains at once, each with its own stream and workspace."""
    cases = [inputs(3, 256, 6000, "e2m1", 1), inputs(20, 512, 4500, "e4m3", 2)]
    want = [serve(*a) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [serve(*a, stream=s) for a, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for p, q in zip(got, want):
            for i, j in zip(p, q):
                assert torch.equal(i, j)


def train(x, res, g, W, t, go, dh, ws=None, rws=None):
    y, rstd, h = vce.rms_forward(x, g, res)
    loss, mean, stats, nv = vce.lce_forward(y, W, t, 0.0, True, -100, workspace=ws)
    dY, dW = vce.lce_backward(y, W, t, stats, nv, go, 0.0, True, -100, workspace=ws)
    dx, dg = vce.rms_backward(dY, h, g, rstd, dh, workspace=rws)
    return y, rstd, h, loss, mean, dY, dW, dx, dg


def train_inputs(M, H, V, seed):
    r = np.random.default_rng(seed)
    t = torch.tensor(r.integers(0, V, M), device="cuda")
    t[::5] = -100
    return (rand((M, H), "bf16", seed), rand((M, H), "bf16", seed + 1),
            1.0 + rand((H,), "fp32", seed + 2, 0.1), rand((V, H), "bf16", seed + 3, H ** -0.5), t,
            torch.full((1,), float(M), device="cuda"), rand((M, H), "bf16", seed + 4))


def whole(x, res, g, W, t, scale):
    """FP64: loss summed over the valid rows times `scale`, and its parts."""
    y, r, h = head.rms_forward(x, g, res, 1e-6)
    z = y @ W.T
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    p = e / e.sum(axis=1, keepdims=True)
    ok = t >= 0
    rows = np.arange(len(t))
    nll = np.where(ok, m[:, 0] + np.log(e.sum(axis=1)) - z[rows, np.where(ok, t, 0)], 0.0)
    d = p.copy()
    d[rows, np.where(ok, t, 0)] -= 1.0
    d *= (ok * scale)[:, None]
    return dict(y=y, r=r, h=h, p=p, loss=nll.sum() * scale, dY=d @ W)


@pytest.mark.parametrize("M,H,V", [(40, 256, 1000), (130, 520, 777)])
def test_training(M, H, V):
    a = train_inputs(M, H, V, M)
    x, res, g, W, t, go, dh = a
    y, rstd, h, loss, mean, dY, dW, dx, dg = train(*a)
    # the norm's gradient on the head's
    rdx, rdg, T, S = head.rms_backward(f64(dY), f64(h), f64(g), f64(rstd), f64(dh))
    assert_within(f64(dx), rdx, HALF[dx.dtype] * np.abs(rdx) + 100 * U * T + TINY, "dx")
    assert_within(f64(dg), rdg, 80 * U * S + TINY, "dweight")
    # the whole, in FP64 from x and the residual on
    tt, nv = t.cpu().numpy(), int((t >= 0).sum())
    scale = float(go.item()) / nv
    R = whole(f64(x), f64(res), f64(g), f64(W), tt, scale)
    edx = head.rms_backward(R["dY"], R["h"], f64(g), R["r"], f64(dh))[0]
    # y is off by half a step of BF16, and by h's (stored in BF16): the norm keeps the
    # relative size; so logits are off by at most dz, the probabilities by a factor
    # exp(2 dz), and the gradient of y by what that moves, its own rounding and the
    # head's (LINEAR_FROB_RTOL of the whole).  The norm's gradient scales a row by rstd
    # and the largest weight at most; h's rounding moves its direction by 2 ||h|| 2^-8.
    half = HALF[torch.bfloat16]
    aW = np.abs(f64(W))
    dz = (1.01 * half * np.abs(R["y"]) @ aW.T).max(axis=1, keepdims=True)
    dp = R["p"] * (np.exp(2 * dz) - 1.0)
    gmax = np.abs(f64(g)).max()
    row = np.linalg.norm(R["dY"], axis=1)
    moved = np.where(tt >= 0, scale * np.linalg.norm(dp @ aW, axis=1), 0.0)
    head_err = LINEAR_FROB_RTOL * np.linalg.norm(R["dY"]) + half * row
    # (1 %: second order.)
    err = 1.01 * (R["r"] * gmax * (moved + head_err + 3 * half * row) +
                  half * np.linalg.norm(edx, axis=1))
    assert np.all(np.linalg.norm(f64(dx) - edx, axis=1) <= err)
    assert rel_frobenius(f64(dx), edx) <= np.linalg.norm(err) / np.linalg.norm(edx)
    # against differences of the FP64 loss along a direction, the residual stream's
    # share <dh, h> included; step 1e-4 leaves an error of its square
    d = np.random.default_rng(1).standard_normal(x.shape)
    f = lambda s: (lambda q: q["loss"] + np.sum(f64(dh) * q["h"]))(
        whole(f64(x) + s * d, f64(res), f64(g), f64(W), tt, scale))
    diff = (f(1e-4) - f(-1e-4)) / 2e-4
    assert abs(np.sum(edx * d) - diff) <= 1e-5 * np.sum(np.abs(edx * d))
    assert abs(np.sum(f64(dx) * d) - diff) <= np.sum(err * np.linalg.norm(d, axis=1)) + \
        1e-5 * np.sum(np.abs(edx * d))


def test_training_graph():
    M, H, V = 70, 264, 900
    a = train_inputs(M, H, V, 3)
    ws = torch.empty(vce.lce_workspace_size(M, H, V), dtype=torch.uint8, device="cuda")
    rws = vce.rms_backward_workspace(M, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        train(*a, ws, rws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = train(*a, ws, rws)
    for i in range(3):
        for old, new in zip(a, train_inputs(M, H, V, 30 + i)):
            old.copy_(new)
        want = train(*a)
        graph.replay()
        torch.cuda.synchronize()
        for n, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), (i, n)
