"""FP32 logits from mx_logits do not depend on other tokens and other rows of W: tokens and rows
of zeros, with a NaN scale or with scales far from 1 leave the logits of the others as they
are, bit for bit, and within K u S of FP64 (every product exact, K additions each off by
at most u of the sum of the terms' sizes S).  A pair with a far-scaled operand goes through the
scaled matrix instructions: 2^-10 G besides, G the sum of its groups' largest products (zero for
two E2M1 operands)."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import TINY, U, assert_within, f64, rand
from oracle import head
from test_parity_mx_logits import PAIRS, group_peaks

pytestmark = pytest.mark.gpu
# up to 16 tokens, tiles of 64, 128 and 256 tokens; K in whole and in broken supersteps
SHAPES = [(3, 70, 64), (16, 130, 544), (9, 65600, 512), (4, 131100, 64), (5, 70, 4640), (40, 300, 96),
          (300, 300, 512), (100, 49300, 256), (130, 49200, 288), (300, 24700, 256),
          (257, 24700, 96)]


def operands(M, V, K, xf, wf):
    X, W = rand((M, K), "bf16", M), rand((V, K), "bf16", V, K ** -0.5)
    X[:, ::97] *= 20
    return [*vce.mx_quantize(X, xf), *vce.mx_quantize(W, wf)]


def values(q, s, fmt):
    return head.dequantize(q.cpu().numpy(), s.cpu().numpy(), fmt)


def same_bits(a, b):
    return torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_zero_nan_and_far_rows(M, V, K, xf, wf):
    args = dict(x_fmt=xf, w_fmt=wf, dtype=torch.float32)
    x, xs, w, ws = operands(M, V, K, xf, wf)
    base = vce.mx_logits(x, xs, w, ws, **args)
    a, b = values(x, xs, xf), values(w, ws, wf)
    ref, S = a @ b.T, np.abs(a) @ np.abs(b).T
    assert_within(f64(base), ref, U * np.abs(ref) + K * U * S, "logits")

    zero_t, nan_t, far_t = M // 2, M - 1, 0
    zero_v, nan_v, far_v = V // 3, 5, V - 1
    x[zero_t], xs[zero_t] = 0, 0
    w[zero_v], ws[zero_v] = 0, 0
    xs[nan_t, K // 64], ws[nan_v, 0] = 255, 255
    if M > 3:
        xs[far_t] -= 90
        ws[far_v] -= 80
    got = vce.mx_logits(x, xs, w, ws, **args)

    assert torch.isnan(got[nan_t]).all() and torch.isnan(got[:, nan_v]).all()
    live_t = torch.ones(M, dtype=torch.bool)
    live_v = torch.ones(V, dtype=torch.bool)
    live_t[nan_t], live_v[nan_v] = False, False
    g = got[live_t.cuda()][:, live_v.cuda()]
    assert not torch.isnan(g).any()
    assert (got[zero_t][live_v.cuda()] == 0).all() and (got[live_t.cuda(), zero_v] == 0).all()
    if M > 3:  # the far token and row: their own error only
        for rows, cols in (([far_t], slice(None)), (slice(None), [far_v])):
            a = np.where(xs.cpu().numpy()[rows].repeat(32, 1) == 255, 0,
                         head.dequantize(x[rows].cpu().numpy(),
                                         xs[rows].cpu().numpy() % 255, xf))
            b = np.where(ws.cpu().numpy()[cols].repeat(32, 1) == 255, 0,
                         head.dequantize(w[cols].cpu().numpy(),
                                         ws[cols].cpu().numpy() % 255, wf))
            r, s = a @ b.T, np.abs(a) @ np.abs(b).T
            out = f64(got[rows][:, cols])
            bound = U * np.abs(r) + K * U * s + K * TINY  # (far by far: below the normal range)
            if "e4m3" in (xf, wf):
                bound += 2.0 ** -10 * group_peaks(a, b)
            assert_within(np.where(np.isnan(out), r, out), r, bound, "far rows")
        live_t[far_t], live_v[far_v] = False, False
    live_t[zero_t], live_v[zero_v] = False, False
    lt, lv = live_t.cuda(), live_v.cuda()
    assert same_bits(got[lt][:, lv].contiguous(), base[lt][:, lv].contiguous())


@pytest.mark.parametrize("xf,wf", PAIRS)
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_zero_blocks(M, V, K, xf, wf):
    """A block of zeros (of either sign) adds nothing, whatever its scale: byte 0, as
    mx_quantize gives it, or the largest, against 127."""
    rng = np.random.default_rng(M + K)
    args = dict(x_fmt=xf, w_fmt=wf, dtype=torch.float32)
    x, xs, w, ws = operands(M, V, K, xf, wf)

    def clear(q, s, fmt, some):
        hit = torch.from_numpy(rng.random(s.shape) < 0.3).cuda()
        hit[some] = False
        n = 32 if fmt == "e4m3" else 16
        zero = torch.from_numpy(rng.integers(0, 2, q.shape).astype(np.uint8) *
                                (0x80 if fmt == "e4m3" else 0x88)).cuda()
        q.copy_(torch.where(hit.repeat_interleave(n, 1), zero, q))
        return hit
    hx, hw = clear(x, xs, xf, M // 2), clear(w, ws, wf, V // 2)
    xs[hx], ws[hw] = 127, 127
    want = vce.mx_logits(x, xs, w, ws, **args)
    a, b = values(x, xs, xf), values(w, ws, wf)
    ref, S = a @ b.T, np.abs(a) @ np.abs(b).T
    assert_within(f64(want), ref, U * np.abs(ref) + K * U * S, "logits")
    for bx, bw in ((0, 127), (127, 0), (0, 0), (254, 3)):
        xs[hx], ws[hw] = bx, bw
        assert same_bits(vce.mx_logits(x, xs, w, ws, **args), want)


@pytest.mark.parametrize("xf,wf", [("e4m3", "e2m1"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("M,V,K", [(1, 1, 32), (2, 5, 32), (13, 333, 608), (17, 1, 32), (70, 301, 288),
                                   (100, 49301, 160), (280, 24701, 128)])
def test_padded_outputs(M, V, K, xf, wf):
    """Far and NaN rows write their own logits only, whatever the output's rows and alignment."""
    x, xs, w, ws = operands(M, V, K, xf, wf)
    args = dict(x_fmt=xf, w_fmt=wf, dtype=torch.float32)
    xs[M - 1] -= 90
    ws[V // 2] -= 80
    if M > 1:
        xs[0, 0] = 255
    ref = vce.mx_logits(x, xs, w, ws, **args)
    assert torch.isnan(ref[0]).all() == (M > 1) and not torch.isnan(ref[1:]).any()
    for ld, off in ((V, 1), (V + 3, 0), (V + 11, 5), ((V + 7) // 4 * 4, 0)):
        buf = torch.full(((M + 1) * ld + 32,), 7.0, device="cuda")
        out = buf.as_strided((M, V), (ld, 1), off)
        vce.mx_logits(x, xs, w, ws, x_fmt=xf, w_fmt=wf, out=out)
        assert same_bits(out.contiguous(), ref)
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask.as_strided((M, V), (ld, 1), off).fill_(False)
        assert (buf[mask] == 7).all()


@pytest.mark.parametrize("M", [5, 300])
def test_graph(M):
    """A captured call finds the far rows of what it is replayed with."""
    V, K = 1500, 544
    x, xs, w, ws = operands(M, V, K, "e4m3", "e2m1")
    kw = dict(dtype=torch.float32)
    clean = xs.clone()
    vce.mx_logits(x, xs, w, ws, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = vce.mx_logits(x, xs, w, ws, **kw)
    base = vce.mx_logits(x, clean, w, ws, **kw)
    for r in range(5):
        xs.copy_(clean)
        if r % 2:
            xs[r, r] = 255
            xs[0] -= 90
        g.replay()
        e = vce.mx_logits(x, xs, w, ws, **kw)
        torch.cuda.synchronize()
        assert same_bits(out, e)
        rest = [i for i in range(M) if not (r % 2 and i in (0, r))]
        assert same_bits(out[rest], base[rest])
