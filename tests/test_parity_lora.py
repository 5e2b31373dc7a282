"""The low-rank adapters, forward and backward, against FP64."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, HALF, TINY, U, assert_within, f64, rand
from oracle import adapters as ref

pytestmark = pytest.mark.gpu
TWO = 2.0 ** -16  # what two BF16 parts leave of a number


def ids(M, n, seed, order="mixed"):
    g = torch.Generator().manual_seed(seed)
    if order == "none":
        t = torch.full((M,), -1)
    elif order == "one":
        t = torch.full((M,), n - 1)
    elif order == "runs":
        t = torch.sort(torch.randint(-1, n, (M,), generator=g)).values
    else:
        t = torch.randint(-2, n + 2, (M,), generator=g)  # some outside: no adapter
    return t.to(torch.int32).cuda()


def inputs(M, H, V, n, r, seed, ldx=None):
    x = rand((M, ldx or H), "bf16", seed)[:, :H]
    return (x, rand((n, r, H), "bf16", seed + 1, H ** -0.5),
            rand((n, V, r), "bf16", seed + 2, r ** -0.5))


def check_forward(x, a, b, k, w=None, base=None, scale=None, dtype="bf16", out=None, **kw):
    M, H = x.shape
    r = a.shape[1]
    y0 = None if base is None else f64(base)
    got = vce.lora_forward(x, a, b, k, w, base=base, scale=scale, dtype=DT[dtype], out=out, **kw)
    kk = k.cpu().numpy()
    kk = np.where((kk < 0) | (kk >= a.shape[0]), -1, kk)
    y, S1, S2 = ref.forward(f64(x), f64(a), f64(b), kk, None if w is None else f64(w), y0,
                            None if scale is None else f64(scale))
    # the shared sum: H additions; the share: H for s (and its scale), its parts (2^-16 for BF16,
    # 2^-23 for FP32 results), r times three additions, one more; and the result's rounding
    parts = TWO if got.dtype == torch.bfloat16 else 2 * U
    bound = HALF[got.dtype] * np.abs(y) + (H + 4) * U * S1 + \
        ((H + 3 * r + 8) * U + parts) * S2 + 2 * U * np.abs(y) + TINY
    assert_within(f64(got), y, bound, "y")
    return got


SHAPES = [(1, 8, 1, 1, 8), (1, 64, 70, 2, 8), (3, 4096, 1001, 3, 16), (16, 512, 300, 5, 24),
          (17, 136, 129, 4, 8), (33, 1000, 513, 2, 40), (64, 2304, 4099, 9, 16),
          (65, 96, 260, 3, 16), (100, 1160, 777, 7, 32), (257, 264, 515, 5, 64),
          (300, 8, 8, 2, 128), (513, 640, 1030, 17, 8), (1, 4096, 66000, 1, 128)]


@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H,V,n,r", SHAPES)
def test_forward(M, H, V, n, r, dtype, order):
    x, a, b = inputs(M, H, V, n, r, M + H)
    k = ids(M, n, V, order)
    scale = torch.rand(n, device="cuda") + 0.5
    w = rand((V, H), "bf16", 7, 2 * H ** -0.5)
    check_forward(x, a, b, k, w, scale=scale, dtype=dtype)
    base = rand((M, V), dtype, 8, 2.0)
    check_forward(x, a, b, k, base=base, scale=scale, dtype=dtype)
    check_forward(x, a, b, k, dtype=dtype)


@pytest.mark.parametrize("M", [1, 40, 70, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_forward_layouts(M, dtype):
    """Padded rows of x, out and base at odd offsets; in place; nothing written beside the rows."""
    H, V, n, r = 200, 333, 4, 16
    x, a, b = inputs(M, H, V, n, r, 3, ldx=216)
    k = ids(M, n, 4)
    w = rand((V, H), "bf16", 5, H ** -0.5)
    for with_base in (False, True):
        buf = torch.full((M * 340 + 9,), 7.0, dtype=DT[dtype], device="cuda")
        out = buf[3:3 + M * 340].view(M, 340)[:, :V]
        base = None
        if with_base:
            base = rand((M, V + 2), dtype, 6)[:, 1:V + 1]
        check_forward(x, a, b, k, None if with_base else w, base=base, dtype=dtype, out=out)
        rest = buf.clone()
        rest[3:3 + M * 340].view(M, 340)[:, :V] = 7.0
        assert bool((rest == 7.0).all())
        if with_base:
            want = out.clone()
            out.copy_(base)
            vce.lora_forward(x, a, b, k, base=out, out=out)
            assert torch.equal(out, want)


@pytest.mark.parametrize("M", [5, 40, 130, 700])
def test_forward_tokens_apart(M):
    """A token's result does not depend on the others' adapters; no adapter leaves the product."""
    H, V, n, r = 256, 300, 6, 16
    x, a, b = inputs(M, H, V, n, r, 1)
    w = rand((V, H), "bf16", 5, H ** -0.5)
    base = rand((M, V), "fp32", 6)
    k = ids(M, n, 2)
    for kw in (dict(w=w, dtype=torch.float32), dict(base=base)):
        mixed = vce.lora_forward(x, a, b, k, **kw)
        plain = vce.lora_forward(x, a, b, ids(M, n, 2, "none"), **kw)
        for i in range(n):
            one = vce.lora_forward(x, a, b, torch.full_like(k, i), **kw)
            assert torch.equal(mixed[k == i], one[k == i])
        none = (k < 0) | (k >= n)
        assert torch.equal(mixed[none], plain[none])
        if "base" in kw:
            assert torch.equal(plain, base)


@pytest.mark.parametrize("M", [6, 40, 130, 300])
def test_forward_not_finite(M):
    """What is not finite in one adapter's weights or one token reaches its own results only."""
    H, V, n, r = 64, 290, 3, 16
    x, a, b = inputs(M, H, V, n, r, 1)
    w = rand((V, H), "bf16", 5, H ** -0.5)
    k = torch.arange(M, dtype=torch.int32, device="cuda") % 4 - 1
    clean = {t: vce.lora_forward(x, a, b, k, w, dtype=t) for t in (torch.bfloat16, torch.float32)}
    b2, x2 = b.clone(), x.clone()
    b2[1, 7, 3], b2[1, 200, 0] = float("inf"), float("nan")
    x2[3, 5] = float("nan")
    for t, want in clean.items():
        for got, bad in ((vce.lora_forward(x, a, b2, k, w, dtype=t), "b"),
                         (vce.lora_forward(x2, a, b, k, w, dtype=t), "x"),
                         (vce.lora_forward(x, a, b2, k, base=want.clone()), "base")):
            hit = torch.zeros((M, V), dtype=torch.bool, device="cuda")
            if bad == "x":
                hit[3] = True
            else:
                hit[:, [7, 200]] = (k == 1).unsqueeze(1)
            assert not bool(got[hit].isfinite().any())
            if bad != "base":
                assert torch.equal(got[~hit], want[~hit]), bad
            else:
                assert bool(got[~hit].isfinite().all())


# ---- backward --------------------------------------------------------------------------

def check_backward(dy, x, a, b, k, w=None, dx_base=None, scale=None, **kw):
    M, H = x.shape
    n, r, V = a.shape[0], a.shape[1], b.shape[1]
    d0 = None if dx_base is None else f64(dx_base)
    kk = k.cpu().numpy()
    kk = np.where((kk < 0) | (kk >= n), -1, kk)
    ref_args = (f64(dy), f64(x), f64(a), f64(b), kk, None if w is None else f64(w), d0,
                None if scale is None else f64(scale))
    got = vce.lora_backward(dy, x, a, b, k, w, dx_base=dx_base, scale=scale, **kw)
    (dx, da, db), (S1, S2, Sa, Sb) = ref.backward(*ref_args)
    two = TWO if dy.dtype == torch.float32 else 0.0
    if got[0] is not None:
        bound = HALF[torch.bfloat16] * np.abs(dx) + ((V + 4) * U + two) * S1 + \
            ((V + 3 * r + 8) * U + TWO) * S2 + 2 * U * np.abs(dx) + TINY
        assert_within(f64(got[0]), dx, bound, "dx")
    # the gradients: the sums for ds or s, their three parts and dy's (3 u each at most), M
    # places and the parts' six or three products
    if got[1] is not None:
        assert_within(f64(got[1]), da, (V + 6 * M + 40) * U * Sa + TINY, "da")
        assert_within(f64(got[2]), db, (H + 6 * M + 40) * U * Sb + TINY, "db")
    return got


@pytest.mark.parametrize("order", ["mixed", "runs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H,V,n,r", SHAPES[:-1] + [(70, 4096, 300, 1, 128), (40, 72, 9000, 2, 72)])
def test_backward(M, H, V, n, r, dtype, order):
    x, a, b = inputs(M, H, V, n, r, M + V)
    dy = rand((M, V), dtype, 9, 0.1)
    k = ids(M, n, H, order)
    scale = torch.rand(n, device="cuda") + 0.5
    check_backward(dy, x, a, b, k, rand((V, H), "bf16", 7, H ** -0.5), scale=scale)
    check_backward(dy, x, a, b, k, dx_base=rand((M, H), "bf16", 8), scale=scale)
    check_backward(dy, x, a, b, k)


@pytest.mark.parametrize("V", [120, 121, 128, 2047])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_backward_layouts(V, dtype):
    """Padded and odd rows of dy and x, what is behind them not read into the sums; outputs given,
    in place; only what is wanted."""
    M, H, n, r = 90, 136, 3, 16
    x, a, b = inputs(M, H, V, n, r, 3, ldx=144)
    w = rand((V, H), "bf16", 7, H ** -0.5)
    k = ids(M, n, 3)
    for pad, skew in ((0, 0), (8, 0), (5, 1)):
        buf = torch.full((skew + M * (V + pad),), float("nan"), dtype=DT[dtype], device="cuda")
        dy = buf[skew:].view(M, V + pad)[:, :V]
        dy.copy_(rand((M, V), dtype, 4, 0.1))
        full = check_backward(dy, x, a, b, k, w)
        dx, da, db = vce.lora_backward(dy, x, a, b, k, w, need_dx=False)
        assert dx is None and torch.equal(da, full[1]) and torch.equal(db, full[2])
        dx, da, db = vce.lora_backward(dy, x, a, b, k, w, need_adapters=False)
        assert da is None and db is None and torch.equal(dx, full[0])
        given = (torch.empty_like(full[0]), torch.full_like(full[1], 7), torch.full_like(full[2], 7))
        check_backward(dy, x, a, b, k, w, out=given)
        assert all(torch.equal(p, q) for p, q in zip(given, full))
        base = rand((M, H), "bf16", 8)
        want = check_backward(dy, x, a, b, k, dx_base=base)[0]
        got = vce.lora_backward(dy, x, a, b, k, dx_base=base, out=(base, None, None))[0]
        assert got is base and torch.equal(base, want)


def test_backward_without_tokens():
    """Adapters without tokens, no token with an adapter, no tokens at all: zero gradients."""
    x, a, b = inputs(50, 64, 99, 5, 8, 1)
    dy, w = rand((50, 99), "bf16", 2), rand((99, 64), "bf16", 3)
    k = torch.full((50,), 3, dtype=torch.int32, device="cuda")
    out = (None, torch.full((5, 8, 64), 7.0, device="cuda"), torch.full((5, 99, 8), 7.0,
                                                                        device="cuda"))
    _, da, db = check_backward(dy, x, a, b, k, w, out=out)
    rest = [0, 1, 2, 4]
    assert not bool(da[rest].any()) and not bool(db[rest].any()) and bool(da[3].any())
    _, da, db = check_backward(dy, x, a, b, k * 0 - 1, w)
    assert not bool(da.any()) and not bool(db.any())
    dx, da, db = vce.lora_backward(dy[:0], x[:0], a, b, k[:0], w)
    assert dx.shape == (0, 64) and not bool(da.any()) and not bool(db.any())
    assert vce.lora_forward(x[:0], a, b, k[:0], w).shape == (0, 99)


def test_gradients_by_differences():
    """The loss sum(y c), in FP64 over stepped inputs, against the analytic gradients' formula."""
    M, H, V, n, r = 5, 16, 11, 2, 8
    x, a, b = inputs(M, H, V, n, r, 2)
    w = rand((V, H), "bf16", 3)
    k = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32, device="cuda")
    scale = torch.tensor([0.7, 1.9], device="cuda")
    c = rand((M, V), "bf16", 4)
    dx, da, db = vce.lora_backward(c, x, a, b, k, w, scale=scale)
    X, A, B, W, C = (f64(t) for t in (x, a, b, w, c))
    kk, S = k.cpu().numpy(), f64(scale)

    def loss(X, A, B):
        return (ref.forward(X, A, B, kk, W, scale=S)[0] * C).sum()
    h = 1e-4  # the loss is at most of second order in each input: central differences are exact
    for t, g, tol in ((X, f64(dx), 2.0 ** -8), (A, f64(da), 1e-5), (B, f64(db), 1e-5)):
        for i in np.ndindex(t.shape):
            old = t[i]
            t[i] = old + h
            up = loss(X, A, B)
            t[i] = old - h
            d = (up - loss(X, A, B)) / (2 * h)
            t[i] = old
            assert abs(d - g[i]) <= tol * abs(d) + 1e-4, i


# ---- calls ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,V", [(70, 17536), (70, 17541), (257, 4352), (1, 9000)])
def test_backward_uneven_parts(M, V, dtype):
    """The sum over V of dy W in parts of which the last is shorter, with the gradients in its grid."""
    H, n, r = 64, 2, 8
    x, a, b = rand((M, H), "bf16", 1), rand((n, r, H), "bf16", 2, 0.1), rand((n, V, r), "bf16", 3)
    w = rand((V, H), "bf16", 4, 0.1)
    k = (torch.arange(M) % 3 - 1).to(torch.int32).cuda()
    check_backward(rand((M, V), dtype, 5, 0.1), x, a, b, k, w)


@pytest.mark.parametrize("M", [7, 50, 90, 400])
def test_captured(M):
    """Forward and backward captured once, replayed over new tokens and adapters."""
    H, V, n, r = 128, 203, 4, 16
    x, a, b = inputs(M, H, V, n, r, 1)
    w, dy, k = rand((V, H), "bf16", 2), rand((M, V), "bf16", 3), ids(M, n, 4)
    y = torch.empty((M, V), dtype=torch.bfloat16, device="cuda")
    grads = vce.lora_backward(dy, x, a, b, k, w)
    ws = vce.lora_forward_workspace(M, H, V, n, r), vce.lora_backward_workspace(M, H, V, n, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vce.lora_forward(x, a, b, k, w, out=y, workspace=ws[0])
        vce.lora_backward(dy, x, a, b, k, w, out=grads, workspace=ws[1])
    for i in range(4):
        x.copy_(rand((M, H), "bf16", 20 + i))
        dy.copy_(rand((M, V), "bf16", 30 + i))
        k.copy_(ids(M, n, 40 + i, ("mixed", "runs", "one", "none")[i]))
        graph.replay()
        want = (vce.lora_forward(x, a, b, k, w),) + vce.lora_backward(dy, x, a, b, k, w)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((y,) + tuple(grads), want)), i


def test_workspaces_hold():
    """No byte beyond the workspaces, whatever they held before."""
    for M, H, V, n, r in ((9, 64, 70, 3, 8), (300, 136, 99, 20, 40), (70, 512, 1000, 1, 16)):
        x, a, b = inputs(M, H, V, n, r, 1)
        k, w = ids(M, n, 2), rand((V, H), "bf16", 3)
        for dtype in ("bf16", "fp32"):
            dy = rand((M, V), dtype, 4)
            want = (vce.lora_forward(x, a, b, k, w),) + vce.lora_backward(dy, x, a, b, k, w)
            sizes = (vce.lora_forward_workspace_size(M, H, V, n, r),
                     vce.lora_backward_workspace_size(M, H, V, n, r, DT[dtype]))
            bufs = [torch.full((s + 512,), 255, dtype=torch.uint8, device="cuda") for s in sizes]
            got = (vce.lora_forward(x, a, b, k, w, workspace=bufs[0][:sizes[0]]),) + \
                vce.lora_backward(dy, x, a, b, k, w, workspace=bufs[1][:sizes[1]])
            assert all(torch.equal(p, q) for p, q in zip(got, want))
            assert all(bool((t[s:] == 255).all()) for t, s in zip(bufs, sizes))


def test_two_streams():
    cases = []
    for M, H, V, n, r in ((300, 512, 1000, 4, 16), (20, 1024, 5000, 8, 8)):
        x, a, b = inputs(M, H, V, n, r, M)
        cases.append((rand((M, V), "bf16", 4), x, a, b, ids(M, n, 2), rand((V, H), "bf16", 3)))
    run = lambda c, s=None: (vce.lora_forward(*c[1:], stream=s),) + \
        vce.lora_backward(*c, stream=s)
    want = [run(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [run(c, s) for c, s in zip(cases, streams)]
        torch.cuda.synchronize()
        for g, v in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, v))
