"""The operators around the head past 2^31 elements and 2^32 bytes: what a call writes behind
those offsets equals what a call over that part alone gives, bit for bit (values
whose sums are exact, or rows that no other row enters)."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from oracle import head

pytestmark = pytest.mark.gpu
TAIL = 2048


def normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def test_rms():
    M, H = (1 << 20) + 77, 2112
    x, res, w = normal((M, H), 1), normal((M, H), 2), normal((H,), 3)
    cuts = [slice(0, TAIL), slice(M - TAIL, M)]
    y, rstd, h = vce.rms_forward(x, w, res)
    q, s, r8, h8 = vce.rms_forward_mx8(x, w, res)
    dx, dw = vce.rms_backward(y, h, w, rstd, res)
    for c in cuts:
        a = vce.rms_forward(x[c], w, res[c])
        b = vce.rms_forward_mx8(x[c], w, res[c])
        d, _ = vce.rms_backward(a[0], a[2], w, a[1], res[c])
        for got, want in ((y, a[0]), (rstd, a[1]), (h, a[2]), (q, b[0]), (s, b[1]), (r8, b[2]),
                          (h8, b[3]), (dx, d)):
            assert torch.equal(got[c], want)
    # dw: sum_rows y (h r), in FP64 a block of rows at a time; FP32 sums of at most 1024 rows
    # a thread, then 4, 64 and 64 shares: 1200 additions and 3 products of at most the terms' sizes
    ref, size = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    for i in range(0, M, 1 << 15):
        t = y[i:i + (1 << 15)].double() * h[i:i + (1 << 15)].double() * \
            rstd[i:i + (1 << 15), None].double()
        ref += t.sum(0)
        size += t.abs().sum(0)
    assert bool(((dw.double() - ref).abs() <= 1300 * 2.0 ** -24 * size).all())


def test_strided_rows_far_apart():
    ld = (1 << 31) + 64
    buf = torch.zeros(ld + 4096, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((2, 4096), (ld, 1))
    x.copy_(normal((2, 4096), 4))
    w = normal((4096,), 5)
    for a, b in zip(vce.rms_forward(x, w), vce.rms_forward(x.contiguous(), w)):
        assert (a is None and b is None) or torch.equal(a, b)
    for a, b in zip(vce.mx_quantize(x), vce.mx_quantize(x.contiguous())):
        assert torch.equal(a, b)
    u = torch.tensor([0.3, 0.9], device="cuda")
    p = torch.full((2,), 0.9, device="cuda")
    assert torch.equal(vce.ce_sample(x, u, top_p=p), vce.ce_sample(x.contiguous(), u, top_p=p))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_mx(fmt):
    rows, K = (1 << 20) + 77, 4096
    x = normal((rows, K), 6)
    q, s = vce.mx_quantize(x, fmt)
    v = vce.mx_dequantize(q, s, fmt)
    for c in (slice(0, TAIL), slice(rows - TAIL, rows)):
        a, b = vce.mx_quantize(x[c], fmt)
        assert torch.equal(q[c], a) and torch.equal(s[c], b)
        assert torch.equal(v[c], vce.mx_dequantize(a, b, fmt))


def integers(rows, K, fmt, seed):
    """Values -2 .. 2 in steps of 1/2 under scales 1 and 2: every sum here is exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = torch.randint(-4, 5, (rows, K), generator=g, device="cuda", dtype=torch.int8)
    x = n.to(torch.bfloat16) / 2
    x[:, ::32] = 6.0 if fmt == "e2m1" else 448.0
    q, s = vce.mx_quantize(x, fmt)
    # the values that set the scale leave again
    if fmt == "e4m3":
        q[:, ::32] = 0
    else:
        q[:, ::16].bitwise_and_(0xf0)
    s.add_(torch.randint(0, 2, s.shape, generator=g, device="cuda", dtype=torch.uint8))
    return q, s


@pytest.mark.parametrize("M,K,V,xf,wf", [
    (4, 4096, (1 << 20) + 77, "e4m3", "e4m3"),       # W past 2^32 bytes, streamed
    (40, 4096, (1 << 20) + 77, "e2m1", "e4m3"),      # by tiles of 64 tokens
    (300, 4096, (1 << 21) + 333, "e4m3", "e2m1"),    # of 256
    (1100, 64, (1 << 21) + 333, "e4m3", "e2m1"),     # logits past 2^32 bytes and 2^31 elements
    (2100000, 64, 1025, "e2m1", "e2m1"),             # many tokens
])
def test_mx_logits(M, K, V, xf, wf):
    x, xs = integers(M, K, xf, 7)
    w, ws = integers(V, K, wf, 8)
    z = vce.mx_logits(x, xs, w, ws, x_fmt=xf, w_fmt=wf)
    n = 200
    for m in (slice(0, min(M, n)), slice(max(M - n, 0), M)):
        for v in (slice(0, n), slice(V - n, V)):
            part = vce.mx_logits(x[m], xs[m], w[v], ws[v], x_fmt=xf, w_fmt=wf)
            assert torch.equal(z[m, v], part)
            a = head.dequantize(x[m].cpu().numpy(), xs[m].cpu().numpy(), xf)
            b = head.dequantize(w[v].cpu().numpy(), ws[v].cpu().numpy(), wf)
            assert torch.equal(part.cpu(), torch.from_numpy(a @ b.T).to(part.dtype))


def test_sample_many_rows():
    N, V = 20011, 128256
    z = normal((N, V), 9)
    g = torch.Generator(device="cuda").manual_seed(10)
    u = torch.rand(N, generator=g, device="cuda")
    pick = lambda a, d: torch.tensor(a, device="cuda", dtype=d)[
        torch.randint(0, len(a), (N,), generator=g, device="cuda")]
    par = [pick([0.0, 0.5, 1.0], torch.float32), pick([0, 0, 40, 1000], torch.int32),
           pick([1.0, 0.9], torch.float32), pick([0.0, 0.05], torch.float32)]
    tok, lp = vce.ce_sample(z, u, *par, with_logprob=True)
    for c in (slice(0, 24), slice(N // 2, N // 2 + 24), slice(N - 24, N)):
        t, l = vce.ce_sample(z[c], u[c], *[p[c] for p in par], with_logprob=True)
        assert torch.equal(tok[c], t) and torch.equal(lp[c], l)


@pytest.mark.parametrize("V", [3000001, 9000001])
def test_sample_long_row(V):
    z = normal((2, V), 11, torch.float32) * 2
    u = [0.2, 0.97]
    zz = z.double().cpu().numpy()
    t = lambda a, d=torch.float32: torch.tensor(a, device="cuda", dtype=d)
    for k, p, mp in ((0, 1.0, 0.0), (50, 0.9, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.01), (6000, 1.0, 0.0)):
        got = vce.ce_sample(z, t(u), None, t([k] * 2, torch.int32), t([p] * 2), t([mp] * 2))
        want = [head.sample(zz[i], float(np.float32(u[i])), 1.0, k, float(np.float32(p)),
                            float(np.float32(mp)))[0] for i in range(2)]
        assert got.tolist() == want, (k, p, mp)
