"""Refusals of the operators around the head, by the C-ABI (fake addresses,
nothing is launched) and by the binding (CPU tensors)."""
import os

import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from vocabulary_cross_entropy_amd import binding

A = 0x7F0000000000  # a fake, 256-byte aligned device address (never touched)
G = 1 << 33         # apart enough for every size below


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from vocabulary_cross_entropy_amd import build
        build.build()
    return binding.lib()


NAN, INF = float("nan"), float("inf")


def rms(L, mx=False, **kw):
    a = dict(x=A, dtype=1, M=4, H=64, ldx=64, res=A + G, ldr=64, w=A + 2 * G, wd=1, w0=0.0,
             eps=1e-6, y=A + 3 * G, s=A + 4 * G, h=A + 5 * G, rstd=A + 6 * G)
    a.update(kw)
    if mx:
        return L.rms_forward_mx8(a["x"], a["dtype"], a["M"], a["H"], a["ldx"], a["res"], a["ldr"],
                                 a["w"], a["wd"], a["w0"], a["eps"], a["y"], a["s"], a["h"],
                                 a["rstd"], None)
    return L.rms_forward(a["x"], a["dtype"], a["M"], a["H"], a["ldx"], a["res"], a["ldr"], a["w"],
                         a["wd"], a["w0"], a["eps"], a["y"], a["h"], a["rstd"], None)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(wd=-1), 2), (dict(M=-1), 1), (dict(M=1 << 31), 1), (dict(H=0), 1),
    (dict(H=32800, ldx=32800, ldr=32800), 7), (dict(eps=-1.0), 1), (dict(eps=NAN), 1),
    (dict(eps=INF), 1), (dict(w0=NAN), 1), (dict(w0=INF), 1), (dict(x=None), 1),
    (dict(w=None), 1), (dict(y=None), 1), (dict(h=None), 1), (dict(ldx=63), 1), (dict(ldr=63), 1),
    (dict(ldx=-64), 1), (dict(ldx=1 << 62), 1), (dict(x=A + 1), 3), (dict(res=A + G + 1), 3),
    (dict(w=A + 2 * G + 1), 3), (dict(h=A + 5 * G + 1), 3), (dict(rstd=A + 6 * G + 2), 3),
    (dict(h=A + 2), 4), (dict(h=A + G, ldr=128), 4), (dict(rstd=A + 2 * G), 4),
    (dict(h=A + 2 * G), 4), (dict(rstd=A + 5 * G + 256), 4), (dict(h=A + G - 64), 4),
])
def test_rms_forward_rejects(L, mx, kw, code):
    assert rms(L, mx, **kw) == code


def test_rms_forward_rejects_its_own(L):
    assert rms(L, y=A + 3 * G + 1) == 3 and rms(L, True, y=A + 3 * G + 2) == 3
    assert rms(L, y=A + 5 * G) == 4 and rms(L, True, y=A, h=A + 5 * G) == 4
    assert rms(L, True, H=48, ldx=48, ldr=48) == 7 and rms(L, True, s=None) == 1
    assert rms(L, True, s=A + 3 * G + 255) == 4
    assert rms(L, M=0) == 0 and rms(L, True, M=0) == 0


def rbwd(L, **kw):
    a = dict(dy=A, h=A + G, dtype=1, M=4, H=64, w=A + 2 * G, wd=1, w0=0.0, rstd=A + 3 * G,
             dh=A + 4 * G, dx=A + 5 * G, dw=A + 6 * G, ws=A + 7 * G, n=1 << 20)
    a.update(kw)
    return L.rms_backward(a["dy"], a["h"], a["dtype"], a["M"], a["H"], a["w"], a["wd"], a["w0"],
                          a["rstd"], a["dh"], a["dx"], a["dw"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=7), 2), (dict(wd=7), 2), (dict(M=-1), 1), (dict(H=-1), 1), (dict(H=40000), 7),
    (dict(w0=INF), 1), (dict(dy=None), 1), (dict(h=None), 1), (dict(w=None), 1),
    (dict(rstd=None), 1), (dict(dx=None), 1), (dict(ws=None), 1), (dict(n=255), 5),
    (dict(ws=A + 7 * G + 8), 3), (dict(dy=A + 1), 3), (dict(dx=A + 5 * G + 1), 3),
    (dict(dw=A + 6 * G + 2), 3), (dict(dh=A + 4 * G + 1), 3), (dict(dx=A + 2), 4),
    (dict(dx=A + 2 * G), 4), (dict(dw=A + 2 * G), 4), (dict(ws=A + G), 4),
    (dict(dw=A + 7 * G), 4), (dict(ws=A + 5 * G), 4),
])
def test_rms_backward_rejects(L, kw, code):
    assert rbwd(L, **kw) == code


def test_rms_workspace_size(L):
    f = L.rms_backward_workspace_size
    assert f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 32769) == 0 and f(1 << 31, 64) == 0
    assert f(0, 64) == 256 and f(16384, 2304) >= 2304 * 4


def mxq(L, **kw):
    a = dict(x=A, dtype=1, rows=4, K=64, ldx=64, fmt=1, q=A + G, s=A + 2 * G)
    a.update(kw)
    return L.mx_quantize(a["x"], a["dtype"], a["rows"], a["K"], a["ldx"], a["fmt"], a["q"],
                         a["s"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 2), (dict(fmt=2), 2), (dict(fmt=-1), 2), (dict(rows=-1), 1), (dict(K=0), 1),
    (dict(K=48), 7), (dict(rows=1 << 60), 1), (dict(rows=1 << 36), 7), (dict(x=None), 1),
    (dict(q=None), 1), (dict(s=None), 1), (dict(ldx=63), 1), (dict(ldx=-1), 1),
    (dict(x=A + 1), 3), (dict(q=A + G + 8), 3), (dict(q=A), 4), (dict(s=A), 4),
    (dict(s=A + G + 127), 4), (dict(ldx=1 << 62), 1),
])
def test_mx_quantize_rejects(L, kw, code):
    assert mxq(L, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=5), 2), (dict(dtype=2), 2), (dict(rows=-4), 1), (dict(K=33), 7), (dict(q=None), 1),
    (dict(s=None), 1), (dict(o=None), 1), (dict(q=A + 4), 3), (dict(o=A + G + 8), 3),
    (dict(o=A), 4), (dict(s=A + G), 4), (dict(rows=1 << 36), 7),
])
def test_mx_dequantize_rejects(L, kw, code):
    a = dict(q=A, s=A + 2 * G, fmt=0, rows=4, K=64, o=A + G, dtype=1)
    a.update(kw)
    assert L.mx_dequantize(a["q"], a["s"], a["fmt"], a["rows"], a["K"], a["o"], a["dtype"],
                           None) == code


X, W = torch.zeros((3, 64)), torch.zeros(64)
GPU_ONLY = (RuntimeError, "GPU only")


@pytest.mark.parametrize("call,exc", [
    (lambda: vce.rms_forward(X, W), RuntimeError),
    (lambda: vce.rms_forward(X.half(), W), TypeError),
    (lambda: vce.rms_forward(X, W.half()), TypeError),
    (lambda: vce.rms_forward(X[0], W), ValueError),
    (lambda: vce.rms_forward(X.t(), W), ValueError),
    (lambda: vce.rms_forward(X, W[:63]), ValueError),
    (lambda: vce.rms_forward(X, torch.zeros(128)[::2]), ValueError),
    (lambda: vce.rms_forward(X, W, X.bfloat16()), ValueError),
    (lambda: vce.rms_forward(X, W, X[:2]), ValueError),
    (lambda: vce.rms_forward(X, W, out=(X.bfloat16(), None, None)), ValueError),
    (lambda: vce.rms_forward(X, W, out=(X,)), ValueError),
    (lambda: vce.rms_forward(X, W, X, out=(None, None, torch.zeros((3, 128))[:, ::2])),
     ValueError),
    (lambda: vce.rms_forward_mx8(X[:, :48], W[:48]), ValueError),
    (lambda: vce.rms_forward_mx8(X, W, out=(X, None, None, None)), ValueError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(3)), RuntimeError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(4)), ValueError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(3).double()), TypeError),
    (lambda: vce.rms_backward(X.bfloat16(), X, W, torch.zeros(3)), ValueError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(3), X[:2]), ValueError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(3), dweight=W.bfloat16()), ValueError),
    (lambda: vce.rms_backward(X, X, W, torch.zeros(3), workspace=torch.zeros(4)), TypeError),
    (lambda: vce.mx_quantize(X), RuntimeError),
    (lambda: vce.mx_quantize(X, "e5m2"), ValueError),
    (lambda: vce.mx_quantize(X.long()), TypeError),
    (lambda: vce.mx_quantize(X[:, :40]), ValueError),
    (lambda: vce.mx_quantize(X[:, :0]), ValueError),
    (lambda: vce.mx_dequantize(X, X), TypeError),
    (lambda: vce.mx_dequantize(X.byte(), torch.zeros((3, 2)).byte(), "e2m1"), ValueError),
    (lambda: vce.mx_dequantize(X.byte(), torch.zeros((3, 2)).byte(), "e4m3"), RuntimeError),
    (lambda: vce.mx_dequantize(X.byte(), torch.zeros((3, 2)).byte(), "e4m3", torch.float16),
     TypeError),
])
def test_binding_rejects(call, exc):
    with pytest.raises(exc):
        call()


def smp(L, **kw):
    a = dict(z=A, dtype=1, d0=2, d1=3, V=1000, ls0=3000, ls1=1000, T=A + G, k=A + 2 * G,
             p=A + 3 * G, mp=A + 4 * G, u=A + 5 * G, tok=A + 6 * G, lp=A + 7 * G, ws=A + 8 * G,
             n=1 << 30)
    a.update(kw)
    return L.ce_sample(a["z"], a["dtype"], a["d0"], a["d1"], a["V"], a["ls0"], a["ls1"], a["T"],
                       a["k"], a["p"], a["mp"], a["u"], a["tok"], a["lp"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(d0=-1), 1), (dict(V=0), 1), (dict(ls0=-1), 1), (dict(ls1=-1), 1),
    (dict(d0=1 << 20, d1=1 << 12), 1), (dict(d0=1 << 40, d1=1 << 40), 1), (dict(V=1 << 31), 7), (dict(d0=1 << 11, d1=1 << 11), 7),
    (dict(ls0=1 << 62), 1), (dict(z=None), 1), (dict(u=None), 1), (dict(tok=None), 1),
    (dict(ws=None), 1), (dict(z=A + 1), 3), (dict(T=A + G + 2), 3), (dict(k=A + 2 * G + 1), 3),
    (dict(p=A + 3 * G + 1), 3), (dict(mp=A + 4 * G + 1), 3), (dict(u=A + 5 * G + 2), 3),
    (dict(tok=A + 6 * G + 4), 3), (dict(lp=A + 7 * G + 2), 3), (dict(ws=A + 8 * G + 128), 3),
    (dict(n=0), 5), (dict(tok=A + 1024), 4), (dict(lp=A + 5 * G), 4), (dict(ws=A + 2 * G), 4),
    (dict(lp=A + 6 * G + 8), 4), (dict(tok=A + 8 * G + 8), 4),
])
def test_ce_sample_rejects(L, kw, code):
    assert smp(L, **kw) == code


def test_ce_sample_sizes(L):
    f = L.ce_sample_workspace_size
    assert f(-1, 10) == 0 and f(1, 0) == 0 and f(1 << 31, 10) == 0 and f(1, 1 << 31) == 0
    assert f(0, 10) > 0 and f(1, 128256) > 0
    assert smp(L, d0=0) == 0


Z, UU = torch.zeros((3, 50)), torch.zeros(3)


@pytest.mark.parametrize("call,exc", [
    (lambda: vce.ce_sample(Z, UU), RuntimeError),
    (lambda: vce.ce_sample(Z.half(), UU), TypeError),
    (lambda: vce.ce_sample(Z[0], UU), ValueError),
    (lambda: vce.ce_sample(Z.t(), torch.zeros(50)), ValueError),
    (lambda: vce.ce_sample(Z, UU[:2]), ValueError),
    (lambda: vce.ce_sample(Z, UU.double()), TypeError),
    (lambda: vce.ce_sample(Z, UU, top_k=UU), TypeError),
    (lambda: vce.ce_sample(Z, UU, top_k=torch.zeros(3, dtype=torch.int64)), TypeError),
    (lambda: vce.ce_sample(Z, UU, top_p=torch.zeros(6)[::2]), ValueError),
    (lambda: vce.ce_sample(Z, UU, out=UU), ValueError),
    (lambda: vce.ce_sample(Z, UU, workspace=UU), TypeError),
])
def test_ce_sample_binding_rejects(call, exc):
    with pytest.raises(exc):
        call()


def gemm(L, **kw):
    a = dict(x=A, xs=A + G, xf=0, w=A + 2 * G, ws=A + 3 * G, wf=1, M=4, K=64, V=100, s=1.0,
             o=A + 4 * G, dtype=1, ldo=100)
    a.update(kw)
    return L.mx_logits(a["x"], a["xs"], a["xf"], a["w"], a["ws"], a["wf"], a["M"], a["K"],
                       a["V"], a["s"], a["o"], a["dtype"], a["ldo"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(xf=2), 2), (dict(wf=-1), 2), (dict(M=-1), 1), (dict(V=-1), 1),
    (dict(K=0), 1), (dict(K=40), 7), (dict(K=(1 << 20) + 32), 7), (dict(M=1 << 31), 7),
    (dict(V=1 << 31, ldo=1 << 31), 7), (dict(s=NAN), 1), (dict(s=INF), 1), (dict(x=None), 1),
    (dict(xs=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(o=None), 1),
    (dict(ldo=99), 1), (dict(ldo=1 << 62), 1), (dict(x=A + 8), 3), (dict(w=A + 2 * G + 4), 3),
    (dict(o=A + 4 * G + 1), 3), (dict(o=A), 4), (dict(o=A + G), 4), (dict(o=A + 2 * G), 4),
    (dict(o=A + 3 * G), 4),
])
def test_mx_logits_rejects(L, kw, code):
    assert gemm(L, **kw) == code


def test_mx_logits_rejects_more_than_a_launch_holds(L):
    b = 1 << 60  # apart enough for every operand
    far = dict(x=A, xs=A + b, w=A + 2 * b, ws=A + 3 * b, o=A + 4 * b, K=32)
    for M, V in ((1, (1 << 30) + 1), (1 << 38, 256), ((1 << 30) + 256, 256), (1 << 20, 1 << 20)):
        assert gemm(L, M=M, V=V, ldo=V, **far) == 7


def test_mx_logits_empty(L):
    assert gemm(L, M=0) == 0 and gemm(L, V=0, ldo=0) == 0


def u8(r, c):
    return torch.zeros((r, c), dtype=torch.uint8)


@pytest.mark.parametrize("call,exc", [
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 32), u8(9, 2)), RuntimeError),
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 64), u8(9, 2)), ValueError),
    (lambda: vce.mx_logits(u8(3, 32), u8(3, 1), u8(9, 32), u8(9, 2)), ValueError),
    (lambda: vce.mx_logits(u8(3, 64), u8(2, 2), u8(9, 32), u8(9, 2)), ValueError),
    (lambda: vce.mx_logits(X, u8(3, 2), u8(9, 32), u8(9, 2)), TypeError),
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 32), u8(9, 2), dtype=torch.float16),
     TypeError),
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 32), u8(9, 2), out=torch.zeros((3, 8))),
     ValueError),
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 32), u8(9, 2),
                           out=torch.zeros((9, 3)).t()), ValueError),
    (lambda: vce.mx_logits(u8(3, 64), u8(3, 2), u8(9, 32), u8(9, 2), x_fmt="fp8"), ValueError),
    (lambda: vce.mx_logits(u8(3, 128)[:, ::2], u8(3, 2), u8(9, 32), u8(9, 2)), ValueError),
])
def test_mx_logits_binding_rejects(call, exc):
    with pytest.raises(exc):
        call()
