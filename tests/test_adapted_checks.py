"""Refusals of the operators of an adapted head, by the C-ABI (fake addresses, nothing is
launched) and by the binding (CPU tensors)."""
import ctypes
import os

import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from vocabulary_cross_entropy_amd import binding

A = 0x7F0000000000  # a fake, 256-byte aligned device address (never touched)
G = 1 << 33         # apart enough for every size below
NAN, INF = float("nan"), float("inf")
GPU_ONLY = (RuntimeError, "GPU only")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(binding.LIB_PATH):
        from vocabulary_cross_entropy_amd import build
        build.build()
    return binding.lib()


# ---- the optimizer step ----------------------------------------------------------

def entry(p=A, g=A + G, n=1000, off=0, pd=1, gd=0):
    return (p, g, n, off, pd | gd << 32)


def adamw(L, entries=(entry(),), **kw):
    a = dict(count=None, bits=8, m=A + 2 * G, v=A + 3 * G, ms=A + 4 * G, vs=A + 5 * G,
             master=A + 6 * G, total=1024, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, step=1,
             lrd=A + 7 * G, std=A + 7 * G + 8, gs=A + 7 * G + 16)
    a.update(kw)
    flat = [x for e in entries for x in e]
    tab = (ctypes.c_int64 * len(flat))(*flat) if entries else None
    return L.adamw_step(tab, len(entries) if a["count"] is None else a["count"], a["bits"],
                        a["m"], a["v"], a["ms"], a["vs"], a["master"], a["total"], a["lr"],
                        a["b1"], a["b2"], a["eps"], a["wd"], a["step"], a["lrd"], a["std"],
                        a["gs"], 7, None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(total=-128), 1), (dict(total=1000), 1), (dict(bits=16), 1),
    (dict(bits=4), 1), (dict(total=1 << 41), 7), (dict(lr=-1.0), 1), (dict(lr=NAN), 1),
    (dict(lr=INF), 1), (dict(eps=-1e-9), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(eps=1e-38), 1), (dict(wd=-0.1), 1), (dict(wd=NAN), 1), (dict(wd=INF), 1), (dict(b1=1.0), 1),
    (dict(b1=-0.1), 1), (dict(b1=NAN), 1), (dict(b2=1.0), 1), (dict(b2=NAN), 1),
    (dict(step=0), 1), (dict(step=-3), 1), (dict(m=None), 1), (dict(v=None), 1),
    (dict(ms=None), 1), (dict(vs=None), 1), (dict(total=0), 1), (dict(total=896), 1),
    (dict(m=A + 2 * G + 8), 3), (dict(v=A + 3 * G + 4), 3), (dict(master=A + 6 * G + 8), 3),
    (dict(lrd=A + 7 * G + 2), 3), (dict(std=A + 7 * G + 4), 3), (dict(gs=A + 7 * G + 1), 3),
    (dict(m=A), 4), (dict(v=A + G), 4), (dict(m=A + 3 * G), 4), (dict(ms=A + 5 * G), 4),
    (dict(vs=A + 2 * G + 1023), 4), (dict(master=A), 4), (dict(lrd=A + 2 * G), 4),
    (dict(std=A + 6 * G + 4088), 4), (dict(gs=A + 1000), 4), (dict(lrd=A + 3 * G + 1020), 4),
])
def test_adamw_rejects(L, kw, code):
    assert adamw(L, **kw) == code


@pytest.mark.parametrize("e,code", [
    ((entry(pd=2),), 2), ((entry(gd=-1),), 2), ((entry(n=-1),), 1), ((entry(p=0),), 1),
    ((entry(g=0),), 1), ((entry(off=-128),), 1), ((entry(off=64),), 1), ((entry(off=128),), 1),
    ((entry(n=1025),), 1), ((entry(n=1 << 62),), 1), ((entry(p=A + 1),), 3),
    ((entry(g=A + G + 2),), 3), ((entry(g=A),), 4), ((entry(g=A + 1996),), 4),
    ((entry(n=100), entry(n=100)), 4),                              # one tensor twice
    ((entry(n=100), entry(p=A + 200, g=A + 2 * G - 400, n=10, off=0)), 4),   # one place
    ((entry(n=129), entry(p=A + 4096, g=A + G + 4096, n=1, off=128)), 4),
    ((entry(n=100), entry(p=A + 198, g=A + G + 400, n=1, off=128)), 4),
    ((entry(n=100), entry(p=A + 200, g=A + 100, n=1, off=128)), 4),  # a gradient in a parameter
])
def test_adamw_rejects_tensors(L, e, code):
    assert adamw(L, e) == code


def test_adamw_nothing_to_do(L):
    assert adamw(L, (), total=0, m=None, v=None, ms=None, vs=None) == 0
    assert adamw(L, (entry(0, 0, 0),), total=0) == 0
    assert adamw(L, (), count=1, total=0) == 1 and adamw(L, (), count=1) == 1
    assert adamw(L, count=(1 << 20) + 1) == 7


def norm(L, entries=((A, 1000, 1),), **kw):
    a = dict(count=len(entries), most=1.0, norm=A + G, scale=A + G + 4, ws=A + 2 * G, n=1 << 16)
    a.update(kw)
    flat = [x for e in entries for x in e]
    tab = (ctypes.c_int64 * len(flat))(*flat) if entries else None
    return L.grad_norm(tab, a["count"], a["most"], a["norm"], a["scale"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(most=0.0), 1), (dict(most=-1.0), 1), (dict(most=NAN), 1),
    (dict(ws=None), 1), (dict(n=7), 5), (dict(norm=A + G + 2), 3), (dict(scale=A + 2), 3),
    (dict(ws=A + 2 * G + 4), 3), (dict(scale=A + G), 4), (dict(norm=A + 1996), 4),
    (dict(ws=A), 4), (dict(norm=A + 2 * G), 4), (dict(entries=((A, -1, 0),)), 1),
    (dict(entries=((0, 5, 0),)), 1), (dict(entries=((A, 5, 2),)), 2),
    (dict(entries=((A + 1, 5, 1),)), 3), (dict(entries=((A, 1 << 41, 0),)), 7),
    (dict(entries=(), count=1), 1), (dict(norm=None, scale=None), 0),
    (dict(count=(1 << 20) + 1), 7),
])
def test_grad_norm_rejects(L, kw, code):
    assert norm(L, **kw) == code


def test_grad_norm_workspace(L):
    f = L.grad_norm_workspace_size
    assert f(-1, 1) == 0 and f(1, -1) == 0 and f(1 << 41, 1) == 0 and f(1, 1 << 21) == 0
    assert f(0, 0) >= 8 and f(1 << 20, 3) >= 64 * 8


P = [torch.zeros(40), torch.zeros((3, 5), dtype=torch.bfloat16)]
BAD_STEP = [
    (dict(params=P[:1]), ValueError, "holds 2"),
    (dict(grads=P[:1]), ValueError, "holds 2"),
    (dict(params=[P[0].double(), P[1]]), TypeError, "float32 or bfloat16"),
    (dict(grads=[P[0].half(), P[1]]), TypeError, "float32 or bfloat16"),
    (dict(params=[torch.zeros(41), P[1]]), ValueError, "size"),
    (dict(grads=[torch.zeros((8, 5)), P[1]]), ValueError, "shape"),
    (dict(grads=[P[0], torch.zeros((5, 3)).t()]), ValueError, "contiguous"),
    (dict(lr=torch.zeros(1, dtype=torch.float64)), TypeError, "lr must be"),
    (dict(lr=torch.zeros(2)), ValueError, "lr must hold 1"),
    (dict(step=torch.zeros(1)), TypeError, "step must be"),
    (dict(grad_scale=torch.zeros(3)), ValueError, "grad_scale must hold 1"),
    (dict(), *GPU_ONLY),
]


@pytest.mark.parametrize("kw,err,text", BAD_STEP)
def test_binding_adamw(kw, err, text):
    a = dict(params=P, grads=P, lr=1e-3, step=1)
    a.update(kw)
    with pytest.raises(err, match=text):
        vce.adamw_step(a.pop("params"), a.pop("grads"), vce.adamw_state(P), a.pop("lr"),
                       a.pop("step"), **a)


def test_binding_adamw_state():
    st = vce.adamw_state(P, 8, True)
    assert st.offsets == [0, 128] and st.sizes == [40, 15] and st.total == 256
    assert st.m.dtype == torch.uint8 and st.m_scales.numel() == 8 and st.master.numel() == 256
    for bad, err in (([], ValueError), ([torch.zeros(3).double()], TypeError),
                     ([torch.zeros((4, 4)).t()[:2]], ValueError)):
        with pytest.raises(err):
            vce.adamw_state(bad)
    with pytest.raises(ValueError):
        vce.adamw_state(P, 16)


def test_binding_grad_norm():
    for grads, kw, err in (([], {}, ValueError), ([None], {}, ValueError),
                           ([P[0].double()], {}, TypeError), ([torch.zeros((4, 6)).t()], {},
                                                              ValueError),
                           (P, dict(out=(torch.zeros(1), None)), ValueError),
                           (P, dict(workspace=torch.zeros(9)), TypeError), (P, {}, RuntimeError)):
        with pytest.raises(err):
            vce.grad_norm(grads, **kw)


# ---- beam search -----------------------------------------------------------------

def bstep(L, **kw):
    a = dict(z=A, dtype=1, B=2, K=3, V=1000, ls0=3000, ls1=1000, s=A + G, ended=A + 2 * G, end=5,
             n=6, score=A + 3 * G, parent=A + 4 * G, token=A + 5 * G, ws=A + 6 * G, wb=1 << 20)
    a.update(kw)
    return L.beam_step(a["z"], a["dtype"], a["B"], a["K"], a["V"], a["ls0"], a["ls1"], a["s"],
                       a["ended"], a["end"], a["n"], a["score"], a["parent"], a["token"],
                       a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 2), (dict(B=-1), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(ls0=-1), 1),
    (dict(ls1=-1), 1), (dict(n=0), 1), (dict(n=257), 7), (dict(K=129), 7),
    (dict(V=(1 << 28) + 1), 7), (dict(B=1 << 22), 7), (dict(B=1 << 21, K=2), 7),
    (dict(end=-1), 1), (dict(end=1000), 1), (dict(z=None), 1), (dict(s=None), 1),
    (dict(score=None), 1), (dict(parent=None), 1), (dict(token=None), 1), (dict(ws=None), 1),
    (dict(ls0=1 << 61), 1), (dict(z=A + 1), 3), (dict(s=A + G + 2), 3),
    (dict(score=A + 3 * G + 2), 3), (dict(parent=A + 4 * G + 1), 3), (dict(token=A + 5 * G + 4), 3),
    (dict(ws=A + 6 * G + 128), 3), (dict(wb=100), 5), (dict(score=A), 4), (dict(parent=A + G), 4),
    (dict(token=A + 2 * G), 4), (dict(ws=A), 4), (dict(parent=A + 3 * G), 4),
    (dict(token=A + 6 * G), 4), (dict(B=0), 0), (dict(ended=None, end=-1, B=0), 0),
])
def test_beam_step_rejects(L, kw, code):
    assert bstep(L, **kw) == code


def test_beam_workspace_size(L):
    f = L.beam_workspace_size
    assert f(-1, 1, 1) == 0 and f(1, 0, 1) == 0 and f(1, 1, 0) == 0 and f(1, 129, 1) == 0
    assert f(0, 4, 10) > 0 and f(2, 3, 8193) >= 2 * f(2, 3, 8192) - 1024


def piece(data=A, inner=64, outer=1, so=0, sk=64, sb=192):
    return (data, inner, outer, so, sk, sb)


def reorder(L, states=(piece(),), **kw):
    a = dict(count=len(states), B=2, K=3, parent=A + G, stride=3)
    a.update(kw)
    flat = [x for e in states for x in e]
    tab = (ctypes.c_int64 * len(flat))(*flat) if states else None
    return L.beam_reorder(tab, a["count"], a["B"], a["K"], a["parent"], a["stride"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(B=-1), 1), (dict(K=0), 1), (dict(stride=-1), 1), (dict(K=129), 7),
    (dict(B=1 << 22), 7), (dict(count=1025), 7), (dict(parent=None), 1), (dict(parent=A + G + 2), 3),
    (dict(stride=1 << 62), 1), (dict(states=(), count=1), 1), (dict(parent=A + 380), 4),
    (dict(states=(piece(inner=-1),)), 1), (dict(states=(piece(outer=-1),)), 1),
    (dict(states=(piece(sk=-64),)), 1), (dict(states=(piece(0),)), 1),
    (dict(states=(piece(inner=1 << 41, sk=1 << 41, sb=1 << 43),)), 7),
    (dict(states=(piece(inner=1 << 39, sk=1 << 39, sb=1 << 41),)), 7),
    (dict(states=(piece(sk=0),)), 4), (dict(states=(piece(sb=0),)), 4),
    (dict(states=(piece(sk=63),)), 4), (dict(states=(piece(sb=191),)), 4),
    (dict(states=(piece(outer=2, so=32),)), 4), (dict(states=(piece(outer=2, so=64),)), 4),
    (dict(states=(piece(sb=1 << 61),)), 1),
    (dict(states=(piece(), piece())), 4),                      # one state twice
    (dict(states=(piece(), piece(A + 320))), 4),               # the last row of one
    (dict(states=(piece(sk=128, sb=384), piece(A + 60, sk=128, sb=384))), 4),
    (dict(states=(piece(sk=128, sb=384), piece(A + 64, 65, sk=128, sb=384))), 4),
    (dict(states=(piece(sk=128, sb=384), piece(A + 64, sk=128, sb=512))), 4),
    (dict(states=(piece(inner=0), piece(0, outer=0)), B=0), 0),
])
def test_beam_reorder_rejects(L, kw, code):
    assert reorder(L, **kw) == code


Z, SC = torch.zeros((2, 3, 50)), torch.zeros((2, 3))
BAD_BEAM = [
    (dict(logits=Z.double()), TypeError, "float32 or bfloat16"),
    (dict(logits=Z[0]), ValueError, r"\(B, K, V\)"),
    (dict(logits=Z.transpose(1, 2)), ValueError, "contiguous"),
    (dict(scores=SC.double()), ValueError, "scores must be"),
    (dict(scores=SC[:1]), ValueError, "scores must be"),
    (dict(ended=torch.zeros((2, 3), dtype=torch.uint8)), ValueError, "ended must be"),
    (dict(out=(None, None)), ValueError, "3 tensors"),
    (dict(out=(None, torch.zeros((2, 3), dtype=torch.int64), None)), ValueError, "parent must be"),
    (dict(workspace=torch.zeros(10)), TypeError, "workspace must be"),
    (dict(), *GPU_ONLY),
]


@pytest.mark.parametrize("kw,err,text", BAD_BEAM)
def test_binding_beam_step(kw, err, text):
    a = dict(logits=Z, scores=SC)
    a.update(kw)
    with pytest.raises(err, match=text):
        vce.beam_step(a.pop("logits"), a.pop("scores"), **a)


PA = torch.zeros((2, 3), dtype=torch.int32)


@pytest.mark.parametrize("states,parent,err,text", [
    ([SC], PA.long(), TypeError, "int32"), ([SC], PA[0], TypeError, "int32"),
    ([SC], PA.t().contiguous().t(), ValueError, "contiguous"),
    ([torch.zeros((2, 4, 5))], PA, ValueError, r"\(2, 3, \.\.\.\)"),
    ([torch.zeros(6)], PA, ValueError, r"\(2, 3, \.\.\.\)"),
    ([torch.zeros((2, 3, 5, 6, 7))[:, :, :3, :4, :5]], PA, ValueError, "equally spaced"),
    ([torch.zeros((2, 3, 5, 6)).transpose(2, 3)], PA, ValueError, "equally spaced"),
    ([SC], PA, *GPU_ONLY),
])
def test_binding_beam_reorder(states, parent, err, text):
    with pytest.raises(err, match=text):
        vce.beam_reorder(states, parent)


def test_beam_pieces():
    f = binding._beam_pieces
    t = torch.zeros((2, 3, 4, 50, 8))
    assert f(t, "t") == (6400, 1, 0, 6400, 19200)
    assert f(t[:, :, :, :33], "t") == (33 * 32, 4, 1600, 6400, 19200)
    assert f(t[:, :, 1:2, :7], "t") == (7 * 32, 1, 0, 6400, 19200)
    assert f(t[..., :3], "t") == (12, 200, 32, 6400, 19200)
    assert f(torch.zeros((2, 3)), "t") == (4, 1, 0, 4, 12)
    assert f(torch.zeros((2, 3, 0, 5)), "t")[0] == 0


# ---- adapters ----------------------------------------------------------------------

def lfwd(L, **kw):
    a = dict(x=A, ldx=64, M=4, H=64, V=100, a=A + G, b=A + 2 * G, n=3, r=16, k=A + 3 * G,
             s=A + 4 * G, w=A + 5 * G, base=None, ldb=0, out=A + 6 * G, dt=1, ldo=100,
             ws=A + 7 * G, wb=1 << 20)
    a.update(kw)
    return L.lora_forward(a["x"], a["ldx"], a["M"], a["H"], a["V"], a["a"], a["b"], a["n"],
                          a["r"], a["k"], a["s"], a["w"], a["base"], a["ldb"], a["out"], a["dt"],
                          a["ldo"], a["ws"], a["wb"], None)


COMMON = [
    (dict(M=-1), 1), (dict(H=0), 1), (dict(V=0), 1), (dict(n=0), 1), (dict(r=0), 1),
    (dict(H=68), 7), (dict(r=12), 7), (dict(r=136), 7), (dict(n=1025), 7),
    (dict(M=(1 << 21) + 1), 7), (dict(H=(1 << 20) + 8), 7), (dict(V=(1 << 22) + 1), 7),
    (dict(dt=2), 2), (dict(ldx=56), 1), (dict(ldx=68), 7), (dict(ldx=(1 << 22) + 8), 7),
    (dict(x=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(k=None), 1), (dict(ws=None), 1),
    (dict(x=A + 8), 3), (dict(a=A + G + 8), 3), (dict(b=A + 2 * G + 2), 3),
    (dict(k=A + 3 * G + 2), 3), (dict(s=A + 4 * G + 1), 3), (dict(w=A + 5 * G + 8), 3),
    (dict(ws=A + 7 * G + 64), 3), (dict(wb=100), 5), (dict(ws=A), 4), (dict(ws=A + 5 * G), 4),
]


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(base=A + 8 * G, ldb=100), 1), (dict(w=None, base=A + 8 * G, ldb=99), 1),
    (dict(ldo=99), 1), (dict(ldo=1 << 62), 1), (dict(out=None), 1), (dict(out=A + 6 * G + 1), 3),
    (dict(w=None, base=A + 8 * G + 1, ldb=100), 3), (dict(out=A), 4), (dict(out=A + G), 4),
    (dict(out=A + 2 * G + 9598), 4), (dict(out=A + 3 * G), 4), (dict(out=A + 4 * G), 4),
    (dict(out=A + 5 * G), 4), (dict(out=A + 7 * G), 4),
    (dict(w=None, base=A + 6 * G, ldb=104, ldo=100), 4),
    (dict(w=None, base=A + 6 * G + 2, ldb=100), 4), (dict(w=None, base=A + 7 * G, ldb=100), 4),
    (dict(M=0), 0), (dict(M=0, x=None, k=None, out=None, ws=None), 0),
])
def test_lora_forward_rejects(L, kw, code):
    assert lfwd(L, **kw) == code


def lbwd(L, **kw):
    a = dict(dy=A + 8 * G, dt=1, ldy=100, x=A, ldx=64, M=4, H=64, V=100, a=A + G, b=A + 2 * G,
             n=3, r=16, k=A + 3 * G, s=A + 4 * G, w=A + 5 * G, base=None, dx=A + 6 * G,
             da=A + 9 * G, db=A + 10 * G, ws=A + 7 * G, wb=1 << 20)
    a.update(kw)
    return L.lora_backward(a["dy"], a["dt"], a["ldy"], a["x"], a["ldx"], a["M"], a["H"], a["V"],
                           a["a"], a["b"], a["n"], a["r"], a["k"], a["s"], a["w"], a["base"],
                           a["dx"], a["da"], a["db"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(base=A + 11 * G), 1), (dict(ldy=99), 1), (dict(ldy=1 << 62), 1), (dict(dy=None), 1),
    (dict(dy=A + 8 * G + 1), 3), (dict(dt=0, dy=A + 8 * G + 2), 3), (dict(dx=A + 6 * G + 8), 3),
    (dict(da=A + 9 * G + 8), 3), (dict(db=A + 10 * G + 4), 3),
    (dict(w=None, base=A + 11 * G + 8), 3), (dict(dx=A + 8 * G), 4), (dict(dx=A), 4),
    (dict(da=A + G), 4), (dict(db=A + 8 * G + 784), 4), (dict(da=A + 10 * G), 4),
    (dict(ws=A + 8 * G), 4), (dict(w=None, base=A + 6 * G + 16), 4),
    (dict(w=None, base=A + 9 * G), 4), (dict(dx=None, da=None, db=None), 0),
    (dict(M=0, da=None, db=None), 0),
])
def test_lora_backward_rejects(L, kw, code):
    assert lbwd(L, **kw) == code


def test_lora_workspace_sizes(L):
    f, g = L.lora_forward_workspace_size, L.lora_backward_workspace_size
    for bad in ((-1, 64, 100, 3, 16), (4, 0, 100, 3, 16), (4, 64, 0, 3, 16), (4, 64, 100, 0, 16),
                (4, 64, 100, 3, 12), (4, 60, 100, 3, 16)):
        assert f(*bad) == 0 and g(*bad, 1) == 0
    assert g(4, 64, 100, 3, 16, 2) == 0
    assert f(0, 64, 100, 3, 16) > 0 and g(0, 64, 100, 3, 16, 1) > 0
    assert g(1000, 64, 4096, 3, 16, 0) >= g(1000, 64, 4096, 3, 16, 1) + 1000 * 4096 * 2


BF = torch.bfloat16
LX, LA, LB = torch.zeros((4, 64), dtype=BF), torch.zeros((3, 16, 64), dtype=BF), \
    torch.zeros((3, 100, 16), dtype=BF)
LK, LW = torch.zeros(4, dtype=torch.int32), torch.zeros((100, 64), dtype=BF)
LY = torch.zeros((4, 100), dtype=BF)
BAD_LORA = [
    (dict(x=LX.float()), TypeError, "x must be bfloat16"),
    (dict(a=LA.float()), TypeError, "a must be bfloat16"),
    (dict(a=LA[:, :, :56].contiguous()), ValueError, "a must be"),
    (dict(b=LB[:2]), ValueError, "a must be"), (dict(b=LB[:, :, :8].contiguous()), ValueError, "a must"),
    (dict(a=LA.transpose(1, 2).contiguous().transpose(1, 2)), ValueError, "a must be contiguous"),
    (dict(k=LK.long()), ValueError, "adapter must be"), (dict(k=LK[:3]), ValueError, "adapter must"),
    (dict(scale=torch.zeros(4)), ValueError, "scale must be"),
    (dict(w=LW[:50]), ValueError, "w must be"), (dict(w=LW.float()), ValueError, "w must be"),
    (dict(workspace=torch.zeros(8)), TypeError, "workspace"),
    (dict(), *GPU_ONLY),
]


@pytest.mark.parametrize("kw,err,text", BAD_LORA + [
    (dict(base=LY), ValueError, "not both"), (dict(dtype=torch.float16), TypeError, "float32 or"),
    (dict(w=None, base=LY.float(), out=LY), ValueError, "base must be"),
    (dict(w=None, base=LY[:, :99]), ValueError, "base must be"),
    (dict(out=LY.t().contiguous().t()), ValueError, "contiguous"),
])
def test_binding_lora_forward(kw, err, text):
    a = dict(x=LX, a=LA, b=LB, k=LK, w=LW)
    a.update(kw)
    with pytest.raises(err, match=text):
        vce.lora_forward(a.pop("x"), a.pop("a"), a.pop("b"), a.pop("k"), a.pop("w"), **a)


@pytest.mark.parametrize("kw,err,text", BAD_LORA + [
    (dict(dx_base=LX), ValueError, "not both"), (dict(dy=LY.half()), TypeError, "dy must be"),
    (dict(dy=LY[:, :99]), ValueError, "dy must be"), (dict(out=(None, None)), ValueError, "3 tensors"),
    (dict(out=(None, LA.float(), LB)), ValueError, "db must be"),
    (dict(w=None, dx_base=LX.float()), ValueError, "dx_base must be"),
])
def test_binding_lora_backward(kw, err, text):
    a = dict(dy=LY, x=LX, a=LA, b=LB, k=LK, w=LW)
    a.update(kw)
    with pytest.raises(err, match=text):
        vce.lora_backward(a.pop("dy"), a.pop("x"), a.pop("a"), a.pop("b"), a.pop("k"),
                          a.pop("w"), **a)
