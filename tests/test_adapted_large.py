"""The operators of an adapted head past 2^31 elements and 2^32 bytes, and at their limits."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import U, f64, rand
from oracle import head, step

pytestmark = pytest.mark.gpu


def test_adapted_logits_past_2_31():
    """M V = 2.2e9 logits, adapters beyond 2^31 elements, by rows against FP32 in torch."""
    M, H, V, n, r = 17000, 64, 130001, 140, 128
    x = rand((M, H), "bf16", 1)
    a = rand((n, r, H), "bf16", 2, H ** -0.5)
    b = torch.empty((n, V, r), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(n):
        b[i] = torch.randn((V, r), generator=g, device="cuda") * r ** -0.5
    w = rand((V, H), "bf16", 4, H ** -0.5)
    k = (torch.arange(M, device="cuda") // 122).to(torch.int32)
    assert b.numel() > 1 << 31 and M * V > 1 << 31
    y = vce.lora_forward(x, a, b, k, w)
    for i in (0, 121, 122, 8000, 16512, 16513, 16999):
        s = x[i].double() @ a[k[i]].double().t()
        want = x[i].double() @ w.double().t() + s @ b[k[i]].double().t()
        # sums of 64 and 128 terms of size one: 2^-8 of the result and 1e-3 of slack
        assert bool(((y[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all()), i
    base = y
    some = torch.tensor([0, 9000, 16999], device="cuda")
    before = base[some].clone()
    vce.lora_forward(x, a, b, k, base=base, out=base)
    for j, i in enumerate(some.tolist()):
        s = x[i].double() @ a[k[i]].double().t()
        want = before[j].double() + s @ b[k[i]].double().t()
        assert bool(((base[i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3).all()), i


@pytest.mark.parametrize("V", [130001, 130048])
def test_adapters_gradients_past_2_31(V):
    """dy of 2.2e9 elements with odd rows, laid out anew, and with rows read in place; the
    gradients of two adapters and some rows of dx."""
    M, H, n, r = 17000, 64, 2, 8
    x, w = rand((M, H), "bf16", 1), rand((V, H), "bf16", 4, H ** -0.5)
    a, b = rand((n, r, H), "bf16", 2, H ** -0.5), rand((n, V, r), "bf16", 3, r ** -0.5)
    dy = torch.empty((M, V), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)
    for i in range(0, M, 1000):
        dy[i:i + 1000] = torch.randn((1000, V), generator=g, device="cuda") * 0.01
    k = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    dx, da, db = vce.lora_backward(dy, x, a, b, k, w)
    wa, wb = torch.zeros((n, r, H), device="cuda").double(), torch.zeros((n, V, r), device="cuda").double()
    for i in range(0, M, 1000):
        d, xx = dy[i:i + 1000].double(), x[i:i + 1000].double()
        for j in range(n):
            on = (k[i:i + 1000] == j).double().unsqueeze(1)
            wa[j] += (on * (d @ b[j].double())).t() @ xx
            wb[j] += d.t() @ (on * (xx @ a[j].double().t()))
    # FP32 sums of some thousand terms of either sign: far below 1e-5 of the whole
    for got, want in ((da, wa), (db, wb)):
        assert ((got.double() - want).norm() / want.norm()).item() <= 1e-5
    for i in (0, 1, 8191, 16998, 16999):
        want = dy[i].double() @ w.double()
        if k[i] >= 0:
            want = want + (dy[i].double() @ b[k[i]].double()) @ a[k[i]].double()
        assert ((dx[i].double() - want).norm() / want.norm()).item() <= 2.0 ** -8, i


@pytest.mark.parametrize("M,n", [(70000, 3), (5000, 1024), (1 << 18, 1000)])
def test_many_tokens_and_adapters(M, n):
    """Tokens beyond what the plan holds in registers, as many adapters as a call takes."""
    H, V, r = 64, 24, 8
    x, a, b = rand((M, H), "bf16", 1), rand((n, r, H), "bf16", 2, 0.1), rand((n, V, r), "bf16", 3)
    k = torch.randint(-1, n, (M,), generator=torch.Generator().manual_seed(4)).to(torch.int32).cuda()
    dy = rand((M, V), "bf16", 5, 0.1)
    y = vce.lora_forward(x, a, b, k)
    dx, da, db = vce.lora_backward(dy, x, a, b, k)
    kk = k.long().clamp(min=0)
    on = (k >= 0).double().unsqueeze(1)
    s = on * torch.bmm(a.double()[kk], x.double().unsqueeze(2)).squeeze(2)
    ds = on * torch.bmm(b.double()[kk].transpose(1, 2).contiguous(), dy.double().unsqueeze(2)).squeeze(2)
    want = torch.bmm(b.double()[kk], s.unsqueeze(2)).squeeze(2)
    assert bool(((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())
    want = torch.bmm(a.double()[kk].transpose(1, 2).contiguous(), ds.unsqueeze(2)).squeeze(2)
    assert bool(((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4).all())
    wa = torch.zeros((n, r, H), dtype=torch.float64, device="cuda")
    wb = torch.zeros((n, V, r), dtype=torch.float64, device="cuda")
    wa.index_add_(0, kk, ds.unsqueeze(2) * x.double().unsqueeze(1))
    wb.index_add_(0, kk, dy.double().unsqueeze(2) * s.unsqueeze(1))
    for got, ref in ((da, wa), (db, wb)):
        assert ((got.double() - ref).norm() / ref.norm()).item() <= 1e-5


def test_step_past_2_32():
    """A parameter of 2^32 + 777 elements in BF16 with 8-bit states: both ends and the seams
    against FP32, with random numbers of the high places; and its gradient's norm."""
    n = (1 << 32) + 777
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    spots = [0, (1 << 31) - 512, (1 << 32) - 512, n - 905]
    r = torch.Generator(device="cuda").manual_seed(1)
    for s in spots:
        p[s:s + 905] = torch.randn(905, generator=r, device="cuda")
        g[s:s + 905] = torch.randn(905, generator=r, device="cuda") * 1e-3
    st = vce.adamw_state([p], 8)
    old = [f64(p[s:s + 905]) for s in spots]
    norm, _ = vce.grad_norm([g])
    want = np.sqrt(sum((f64(g[s:e]) ** 2).sum() for s, e in
                       zip(spots, [905, spots[1] + 905, spots[3], n])))
    assert abs(norm.item() - want) <= 2 * U * want
    vce.adamw_step([p], [g], st, 1e-3, 5, seed=9)
    for s, o in zip(spots, old):
        lo, hi = s // 32 * 32, (s + 905 + 31) // 32 * 32
        gg = torch.zeros(hi - lo, device="cuda")
        e = min(hi, n)
        gg[:e - lo] = g[lo:e].float()
        a, b = step.moments32(gg.cpu().numpy(), 1.0, 0 * gg.cpu().numpy(), 0 * gg.cpu().numpy(),
                              0.9, 0.999)
        bits = step.random_bits(np.arange(lo, hi), 9, 5)
        for x, q, sc, r16, keep in ((a, st.m, st.m_scales, bits & np.uint64(65535), False),
                                    (np.sqrt(b), st.v, st.v_scales, bits >> np.uint64(16), True)):
            code, scale = step.round_random(x, r16, keep)
            assert np.array_equal(q[lo:hi].cpu().numpy(), code), s
            assert np.array_equal(sc[lo // 32:hi // 32].cpu().numpy(), scale), s
        w, _, _ = step.adamw(o, f64(g[s:s + 905]), 0, 0, 1e-3, 5)
        assert (np.abs(f64(p[s:s + 905]) - w) <= 2.0 ** -8 * np.abs(w) + 1e-7).all(), s
    # elsewhere nothing was there to move
    assert not bool(p[10000:20000].any()) and not bool(st.m[10000:20000].any())
