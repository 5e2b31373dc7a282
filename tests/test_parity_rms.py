"""Residual + RMS norm (forward, forward into microscaled 8 bits, backward)
against the FP64 reference.

Bounds.  A row's sum of squares is at most 64 chained FP32 additions a lane
and 20 across lanes, all of positive terms: relative error at most 84 u; the
root halves it; the mean, the root, the reciprocal, the residual's addition
and the products add at most 10 u more: 52 u, taken as C = 64 u.  In the
backward every term of dx passes at most as many additions (inside the mean)
plus the error of rstd (given) and 8 products: 100 u of the terms' sizes.  A
share of dw is at most 8 rows a thread here, 4 wavefronts, 32 shares a lane
and 16 lanes: 60 additions and 3 products, taken as 80 u of the terms' sizes.
"""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, HALF, TINY, U, assert_within, f64, rand
from oracle import head

pytestmark = pytest.mark.gpu
C = 64 * U

SHAPES = [(1, 1), (3, 7), (5, 32), (1, 100), (1030, 64), (4, 512), (1100, 520), (7, 1000),
          (1025, 2304), (9, 2305), (2, 2561), (1024, 4096), (3, 4104), (2, 4097), (3, 8192),
          (2, 8200), (2, 8193), (3, 16384), (2, 16390), (2, 32768), (1, 32767)]


def check_forward(x, w, res, w0, eps, out):
    y, rstd, h = out
    ry, rr, rh = head.rms_forward(f64(x), f64(w), None if res is None else f64(res), eps, w0)
    assert_within(f64(rstd), rr, C * rr, "rstd")
    assert_within(f64(y), ry, (HALF[y.dtype] + C) * np.abs(ry) + TINY, "y")
    if res is None:
        assert h is None
    else:
        assert_within(f64(h), rh, (HALF[h.dtype] + U) * np.abs(rh) + TINY, "h")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_forward(M, H, dtype):
    x, res = rand((M, H), dtype, 1), rand((M, H), dtype, 2, 2.0)
    wd = "fp32" if H % 3 == 0 else dtype
    w = rand((H,), wd, 3)
    check_forward(x, w, res, 1.0, 1e-6, vce.rms_forward(x, w, res, 1e-6, weight_offset=1.0))
    check_forward(x, w, None, 0.0, 1e-3, vce.rms_forward(x, w, None, 1e-3))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_backward(M, H, dtype):
    h, dy = rand((M, H), dtype, 4), rand((M, H), dtype, 5)
    dh = rand((M, H), dtype, 6) if M % 2 else None
    w = rand((H,), "bf16" if H % 3 == 0 else dtype, 7)
    _, rstd, _ = vce.rms_forward(h, w)
    dx, dw = vce.rms_backward(dy, h, w, rstd, dh, weight_offset=1.0)
    rdx, rdw, T, S = head.rms_backward(f64(dy), f64(h), f64(w), f64(rstd),
                                       None if dh is None else f64(dh), 1.0)
    assert_within(f64(dx), rdx, HALF[dx.dtype] * np.abs(rdx) + 100 * U * T + TINY, "dx")
    assert dw.dtype == torch.float32
    assert_within(f64(dw), rdw, 80 * U * S + TINY, "dw")
    again = vce.rms_backward(dy, h, w, rstd, dh, weight_offset=1.0)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only = vce.rms_backward(dy, h, w, rstd, dh, weight_offset=1.0, need_dweight=False)
    assert torch.equal(only[0], dx) and only[1] is None


def test_backward_many_rows():
    M, H = 4099, 96
    h, dy, w = rand((M, H), "fp32", 8), rand((M, H), "fp32", 9), rand((H,), "fp32", 10)
    _, rstd, _ = vce.rms_forward(h, w)
    dx, dw = vce.rms_backward(dy, h, w, rstd)
    rdx, rdw, T, S = head.rms_backward(f64(dy), f64(h), f64(w), f64(rstd))
    assert_within(f64(dx), rdx, HALF[dx.dtype] * np.abs(rdx) + 100 * U * T, "dx")
    assert_within(f64(dw), rdw, 80 * U * S, "dw")


def check_mx8(x, w, res, w0, out):
    """Scales: the least that holds the row's block, to C of its largest value.
    Values: half a step of the grid of the block's scale, and C of the value."""
    q, s, rstd, _ = out
    ry, rr, _ = head.rms_forward(f64(x), f64(w), None if res is None else f64(res), 1e-6, w0)
    M, H = ry.shape
    amax = np.max(np.abs(ry).reshape(M, H // 32, 32), axis=2)
    sb = s.cpu().numpy().astype(int)
    lo, hi = (head.scale_bytes(amax * (1 + k), "e4m3") for k in (-C, C))
    assert np.all((sb >= lo) & (sb <= hi)), "scales"
    v = head.dequantize(q.cpu().numpy(), s.cpu().numpy(), "e4m3")
    sc = np.repeat(2.0 ** (sb - 127.0), 32, axis=1)
    step = head.step_at(np.maximum(np.abs(v), np.abs(ry)), sc, "e4m3")
    assert_within(v, ry, step / 2 + C * np.abs(ry), "values")
    assert_within(f64(rstd), rr, C * rr, "rstd")
    assert_within(f64(vce.mx_dequantize(q, s, "e4m3")), v, 0, "dequantized")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H", [(1, 32), (5, 96), (1100, 512), (3, 2304), (1025, 4096),
                                 (2, 8192), (2, 16384), (1, 32768)])
def test_forward_mx8(M, H, dtype):
    x, res, w = rand((M, H), dtype, 11, 3.0), rand((M, H), dtype, 12), rand((H,), dtype, 13)
    out = vce.rms_forward_mx8(x, w, res, weight_offset=1.0)
    check_mx8(x, w, res, 1.0, out)
    y, rstd, h = vce.rms_forward(x, w, res, weight_offset=1.0)
    assert torch.equal(out[3], h) and torch.equal(out[2], rstd)
    check_mx8(x, w, None, 0.0, vce.rms_forward_mx8(x, w))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strided_rows(dtype):
    """The last token of every sequence, odd strides, one row read many times."""
    H = 96
    full = rand((6, 5, H), dtype, 14)
    last = full[:, -1]
    w = rand((H,), dtype, 15)
    big = rand((6, H + 3), dtype, 16)
    odd = big[:, 1:1 + H]
    one = full[0, :1].expand(6, H)
    for x in (last, odd, one):
        for res in (None, last, odd, one):
            got = vce.rms_forward(x, w, res)
            ref = vce.rms_forward(x.contiguous(), w, None if res is None else res.contiguous())
            check_forward(x, w, res, 0.0, 1e-6, got)
            gq = vce.rms_forward_mx8(x, w, res)
            check_mx8(x, w, res, 0.0, gq)
            assert res is None or torch.equal(got[2], ref[2])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("M,H", [(3, 100), (1100, 2304), (2, 8200)])
def test_in_place(M, H, dtype):
    x, res, w = rand((M, H), dtype, 17), rand((M, H), dtype, 18), rand((H,), dtype, 19)
    y, r, h = vce.rms_forward(x, w, res)
    x2, res2 = x.clone(), res.clone()
    vce.rms_forward(x2, w, res2, out=(x2, None, res2))  # y over x, h over the residual
    assert torch.equal(x2, y) and torch.equal(res2, h)
    dy, dh = rand((M, H), dtype, 20), rand((M, H), dtype, 21)
    dx, dw = vce.rms_backward(dy, h, w, r, dh)
    for k in range(3):
        t = [dy.clone(), h.clone(), dh.clone()]
        gx, gw = vce.rms_backward(t[0], t[1], w, r, t[2], dx=t[k])
        assert torch.equal(gx, dx) and torch.equal(gw, dw)


def test_rows_around_are_left_alone():
    M, H = 5, 96
    x, w = rand((M, H), "bf16", 22), rand((H,), "bf16", 23)
    buf = torch.full((M + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    vce.rms_forward(x, w, out=(buf[1:M + 1], None, None))
    assert (buf[0] == 7).all() and (buf[M + 1] == 7).all()
    q = torch.full((M + 2, H), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 2, H // 32), 9, dtype=torch.uint8, device="cuda")
    vce.rms_forward_mx8(x, w, out=(q[1:M + 1], s[1:M + 1], None, None))
    for t in (q, s):
        assert (t[0] == 9).all() and (t[M + 1] == 9).all()


def test_empty_and_special_rows():
    w = rand((64,), "fp32", 24)
    e = torch.empty((0, 64), device="cuda")
    y, r, h = vce.rms_forward(e, w, e)
    assert y.shape == (0, 64) and h.shape == (0, 64) and r.shape == (0,)
    dx, dw = vce.rms_backward(e, e, w, r)
    assert dx.shape == (0, 64) and (dw == 0).all()
    q, s, _, _ = vce.rms_forward_mx8(e, w)
    assert q.shape == (0, 64) and s.shape == (0, 2)
    x = torch.zeros((4, 64), device="cuda")
    x[1, 3], x[2, 5], x[3] = float("nan"), float("inf"), 1e-30
    y, r, _ = vce.rms_forward(x, w)
    ry, rr, _ = head.rms_forward(f64(x), f64(w))
    assert (y[0] == 0).all() and y[1].isnan().all() and y[2, 5].isnan()
    assert_within(f64(y[3]), ry[3], (C + U) * np.abs(ry[3]), "tiny row")
    q, s, _, _ = vce.rms_forward_mx8(x, w)
    assert s[0].eq(0).all() and s[1].eq(255).all() and s[2, 0] == 255
    assert q[0].bitwise_and(127).eq(0).all() and q[1].eq(0).all()


def test_streams_and_graph():
    """Two streams at once, and a captured step replayed with new inputs."""
    M, H = 700, 2304
    x, res, w = rand((M, H), "bf16", 25), rand((M, H), "bf16", 26), rand((H,), "bf16", 27)
    ref = vce.rms_forward(x, w, res)
    rb = vce.rms_backward(ref[0], ref[2], w, ref[1], res)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[vce.rms_forward(x, w, res, stream=s) for s in (a, b)] for _ in range(3)]
    gb = [[vce.rms_backward(ref[0], ref[2], w, ref[1], res, stream=s) for s in (a, b)]
          for _ in range(3)]
    torch.cuda.synchronize()
    for o in sum(got, []):
        assert all(torch.equal(i, j) for i, j in zip(o, ref))
    for o in sum(gb, []):
        assert all(torch.equal(i, j) for i, j in zip(o, rb))
    xs, rs = x.clone(), res.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, r, h = vce.rms_forward(xs, w, rs)
        dx, dw = vce.rms_backward(y, h, w, r, rs)
        q, s, _, _ = vce.rms_forward_mx8(xs, w, rs)
    for k in range(4):
        xs.copy_(rand((M, H), "bf16", 30 + k))
        g.replay()
        e = vce.rms_forward(xs, w, rs)
        eb = vce.rms_backward(e[0], e[2], w, e[1], rs)
        em = vce.rms_forward_mx8(xs, w, rs)
        torch.cuda.synchronize()
        for i, j in zip((y, r, h, dx, dw, q, s), e + eb + em[:2]):
            assert torch.equal(i, j), k
