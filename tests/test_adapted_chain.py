"""The operators of an adapted head run together with those around it: a fine-tuning step (adapted
logits, loss, adapters' gradients, clipping, AdamW) and beam search with adapters beside a
microscaled head, each stage against its FP64 reference on the stage's own input, whole steps captured,
and the gradients of the whole against autograd."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import HALF, TINY, U, assert_within, f64, rand
from oracle import adapters, beam, head, step

pytestmark = pytest.mark.gpu
M, H, V, N, R = 96, 128, 301, 3, 16


class Head:
    """An adapted head in training: BF16 adapters with FP32 masters, W frozen."""

    def __init__(self, bits, seed=1):
        self.w = rand((V, H), "bf16", seed, H ** -0.5)
        self.a = rand((N, R, H), "bf16", seed + 1, H ** -0.5)
        self.b = rand((N, V, R), "bf16", seed + 2, 0.02)
        self.scale = torch.full((N,), 2.0, device="cuda")
        self.state = vce.adamw_state([self.a, self.b], bits, master=True)
        self.lr = torch.tensor(1e-3, device="cuda")
        self.step = torch.ones(1, dtype=torch.int64, device="cuda")
        e = lambda *s, d=torch.float32: torch.empty(s, dtype=d, device="cuda")
        self.y = e(M, V, d=torch.bfloat16)
        self.dy = e(M, V, d=torch.bfloat16)
        self.grads = (e(M, H, d=torch.bfloat16), e(N, R, H), e(N, V, R))
        self.norm = (e(), e())
        self.ws = (vce.lora_forward_workspace(M, H, V, N, R),
                   vce.lora_backward_workspace(M, H, V, N, R),
                   torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
        self.loss = (e(1, M), e(), e(1, M, 4), e(d=torch.int32))
        self.one = torch.ones(1, device="cuda")

    def train(self, x, k, t, stream=None):
        vce.lora_forward(x, self.a, self.b, k, self.w, scale=self.scale, out=self.y,
                         workspace=self.ws[0], stream=stream)
        vce.ce_forward(self.y[None], t, 0.1, True, out=self.loss, stream=stream)
        vce.ce_backward(self.y[None], t, self.loss[2], self.loss[3], self.one, 0.1, True,
                        grad=self.dy.view(1, M, V), stream=stream)
        vce.lora_backward(self.dy, x, self.a, self.b, k, self.w, scale=self.scale,
                          out=self.grads, workspace=self.ws[1], stream=stream)
        vce.grad_norm(self.grads[1:], 0.01, out=self.norm, workspace=self.ws[2], stream=stream)
        vce.adamw_step([self.a, self.b], self.grads[1:], self.state, self.lr, self.step,
                       grad_scale=self.norm[1], seed=3, stream=stream)

    def tensors(self):
        s = self.state
        return [t for t in (self.a, self.b, self.y, self.dy, *self.grads, *self.norm, s.m, s.v,
                            s.master, s.m_scales, s.v_scales) if t is not None]


def batch(seed):
    g = torch.Generator().manual_seed(seed)
    return (rand((M, H), "bf16", seed),
            torch.randint(-1, N, (M,), generator=g).to(torch.int32).cuda(),
            torch.randint(0, V, (1, M), generator=g).cuda())


@pytest.mark.parametrize("bits", [8, 32])
def test_training_step(bits):
    h = Head(bits)
    x, k, t = batch(7)
    a0, b0, master = h.a.clone(), h.b.clone(), h.state.master.clone()
    h.train(x, k, t)
    kk = k.cpu().numpy()
    args = (f64(x), f64(a0), f64(b0), kk)
    y, S1, S2 = adapters.forward(*args, f64(h.w), None, f64(h.scale))
    assert_within(f64(h.y), y, HALF[h.y.dtype] * np.abs(y) + (H + 4) * U * S1 +
                  ((H + 3 * R + 8) * U + 2.0 ** -16) * S2 + 2 * U * np.abs(y), "logits")
    # the gradients by autograd in float64 from the stored logits' gradient, and of the whole
    X, A, B = (torch.tensor(v, requires_grad=True) for v in args[:3])
    W = torch.tensor(f64(h.w))
    rows = []
    for i in range(M):
        q = W @ X[i]
        rows.append(q + 2.0 * (B[kk[i]] @ (A[kk[i]] @ X[i])) if kk[i] >= 0 else q)
    Y = torch.stack(rows)
    loss = torch.nn.functional.cross_entropy(Y, t.cpu().view(-1), label_smoothing=0.1)
    # a row's loss moves by twice its logits' largest error at most
    delta = np.abs(f64(h.y) - y).max()
    assert abs(loss.item() - h.loss[1].item()) <= 2 * delta + 1e-5 * loss.item()
    loss.backward()
    # a probability by a factor of exp(2 delta), dy by its rounding; from there everything is
    # linear in dy (FP32 sums, 2^-7 of dx for its rounding and two parts)
    p = torch.softmax(Y.detach(), 1).numpy()
    err = 2.0 ** -8 * np.abs(f64(h.dy)) + np.expm1(2 * delta) * p / M + 1e-5 * p / M
    off, _ = adapters.backward(err, *(np.abs(v) for v in args[:3]), kk, np.abs(f64(h.w)), None,
                               f64(h.scale))
    for got, want, e, rel in zip(h.grads, (X, A, B), off, (2.0 ** -7, 1e-4, 1e-4)):
        want = want.grad.numpy()
        assert_within(f64(got), want, e * 1.01 + rel * np.abs(want) + 1e-7, "gradient of the loss")
    ref, sums = adapters.backward(f64(h.dy), *args, f64(h.w), None, f64(h.scale))
    for got, want, S, n in zip(h.grads[1:], ref[1:], sums[2:], (V, H)):
        assert_within(f64(got), want, (n + 6 * M + 40) * U * S + TINY, "adapters' gradients")
    norm = np.sqrt(sum((f64(g) ** 2).sum() for g in h.grads[1:]))
    assert abs(h.norm[0].item() - norm) <= 2 * U * norm
    scale = min(1.0, 0.01 / norm)
    assert abs(h.norm[1].item() - scale) <= 2 * U * scale
    for i, (p, g) in enumerate(zip((h.a, h.b), h.grads[1:])):
        o, n = h.state.offsets[i], h.state.sizes[i]
        old, gg = f64(master[o:o + n]), f64(g).reshape(-1) * scale
        want, _, _ = step.adamw(old, gg, 0, 0, 1e-3, 1)
        # first step: lr sign(g) where |g| is above eps, plus decay; its own error 30 u of lr
        bound = 4 * U * np.abs(old) + 30 * U * 1e-3 + TINY
        assert_within(f64(h.state.master[o:o + n]), want, bound, "master")
        assert_within(f64(p).reshape(-1), want, HALF[p.dtype] * (np.abs(want) + bound) + bound, "p")


@pytest.mark.parametrize("bits", [8, 32])
def test_training_captured(bits):
    """A whole step captured once and replayed over new batches, rates and step numbers."""
    graphed, eager = Head(bits), Head(bits)
    x, k, t = batch(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphed.train(x, k, t, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    eager.train(x, k, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.train(x, k, t)
    for i in range(5):
        for old, new in zip((x, k, t), batch(20 + i)):
            old.copy_(new)
        for h in (graphed, eager):
            h.step.fill_(i + 2)
            h.lr.fill_(1e-3 / (i + 1))
        graph.replay()
        eager.train(x, k, t)
        torch.cuda.synchronize()
        for n, (p, q) in enumerate(zip(graphed.tensors(), eager.tensors())):
            assert torch.equal(p, q), (i, n)


def test_beam_search_with_adapters():
    """Norm to 8 bits, microscaled logits, the requests' adapters beside them, a beam step, states
    reordered; three steps, each against its reference, then captured."""
    B, K, Vs, Hs = 4, 4, 1001, 256
    w, ws = vce.mx_quantize(rand((Vs, Hs), "bf16", 1, Hs ** -0.5), "e4m3")
    g = rand((Hs,), "bf16", 2, 0.1)
    a, b = rand((N, 8, Hs), "bf16", 3, Hs ** -0.5), rand((N, Vs, 8), "bf16", 4, 0.3)
    k = torch.tensor([0, -1, 2, 1], dtype=torch.int32, device="cuda").repeat_interleave(K)
    work = vce.lora_forward_workspace(B * K, Hs, Vs, N, 8), vce.beam_workspace(B, K, Vs)
    scores = torch.full((B, K), -float("inf"), device="cuda")
    scores[:, 0] = 0.0  # one beam to begin with
    hist = torch.zeros((B, K, 3), dtype=torch.int64, device="cuda")
    cache = torch.randn((B, K, 5, 20, 8), device="cuda")
    x, res = (rand((B * K, Hs), "bf16", s) for s in (5, 6))
    z = torch.empty((B * K, Vs), dtype=torch.float32, device="cuda")
    out = (torch.empty((B, K), device="cuda"),
           torch.empty((B, K), dtype=torch.int32, device="cuda"),
           torch.empty((B, K), dtype=torch.int64, device="cuda"))
    norm = (torch.empty((B * K, Hs), dtype=torch.uint8, device="cuda"),
            torch.empty((B * K, Hs // 32), dtype=torch.uint8, device="cuda"),
            torch.empty(B * K, device="cuda"),
            torch.empty((B * K, Hs), dtype=torch.bfloat16, device="cuda"))

    def one(h, c):
        q, s, _, r = vce.rms_forward_mx8(x, g, res, weight_offset=1.0, out=norm)
        vce.mx_logits(q, s, w, ws, w_fmt="e4m3", out=z)
        # the adapters take the residual stream in BF16
        vce.lora_forward(r, a, b, k, base=z, out=z, workspace=work[0])
        vce.beam_step(z.view(B, K, Vs), scores, workspace=work[1], out=out)
        vce.beam_reorder([h, c[:, :, :, :13]], out[1])

    def check(h, c, h0, c0, s0):
        zz = f64(z).reshape(B, K, Vs)
        for i in range(B):
            v, p, t = beam.step(zz[i], f64(s0)[i], K)
            assert out[1][i].tolist() == p.tolist() and out[2][i].tolist() == t.tolist()
            assert np.allclose(f64(out[0])[i], v, rtol=U, atol=2e-11)
            assert torch.equal(h[i], h0[i][out[1][i].long()])
            assert torch.equal(c[i][:, :, :13], c0[i][out[1][i].long()][:, :, :13])
        assert torch.equal(c[:, :, :, 13:], c0[:, :, :, 13:])

    for i in range(3):
        h0, c0, s0 = hist.clone(), cache.clone(), scores.clone()
        one(hist, cache)
        y = head.dequantize(norm[0].cpu().numpy(), norm[1].cpu().numpy(), "e4m3")
        wd = head.dequantize(w.cpu().numpy(), ws.cpu().numpy(), "e4m3")
        want, S1, S2 = adapters.forward(f64(norm[3]), f64(a), f64(b), k.cpu().numpy(), None,
                                        y @ wd.T)
        S = np.abs(y) @ np.abs(wd).T
        # exact products, FP32 sums of H terms; the share as in its own tests
        assert_within(f64(z), want, (Hs + 4) * U * S + ((Hs + 32) * U + 2 * U) * S2 +
                      4 * U * np.abs(want), "logits")
        check(hist, cache, h0, c0, s0)
        hist[:, :, i] = out[2]
        scores.copy_(out[0])
        x.copy_(rand((B * K, Hs), "bf16", 30 + i))
    h2, c2 = hist.clone(), cache.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one(h2, c2)
    h2.copy_(hist), c2.copy_(cache)
    for i in range(4):
        h0, c0 = h2.clone(), c2.clone()
        x.copy_(rand((B * K, Hs), "bf16", 50 + i))
        graph.replay()
        torch.cuda.synchronize()
        check(h2, c2, h0, c0, scores)
        got = [t.clone() for t in out]
        hist.copy_(h0), cache.copy_(c0)
        one(hist, cache)
        assert all(torch.equal(p, q) for p, q in zip(got, out)) and torch.equal(hist, h2)
        assert torch.equal(cache, c2)


def test_draw_with_adapters():
    """A token per row from adapted logits: the adapters' share on top of the microscaled head's
    BF16 logits in place, then the draw."""
    Vs, Hs, n = 5003, 512, 20
    w, ws = vce.mx_quantize(rand((Vs, Hs), "bf16", 1, Hs ** -0.5), "e2m1")
    x = rand((n, Hs), "bf16", 2)
    q, s = vce.mx_quantize(x, "e4m3")
    z = vce.mx_logits(q, s, w, ws)
    a, b = rand((N, R, Hs), "bf16", 3, Hs ** -0.5), rand((N, Vs, R), "bf16", 4, 0.3)
    k = (torch.arange(n, device="cuda") % (N + 1) - 1).to(torch.int32)
    plain = z.clone()
    vce.lora_forward(x, a, b, k, base=z, out=z)
    want, _, S2 = adapters.forward(f64(x), f64(a), f64(b), k.cpu().numpy(), None, f64(plain))
    assert_within(f64(z), want, (HALF[z.dtype] + 2 * U) * np.abs(want) +
                  ((Hs + 3 * R + 8) * U + 2.0 ** -16) * S2, "logits")
    assert torch.equal(z[k < 0], plain[k < 0])
    u = torch.rand(n, device="cuda")
    tok = vce.ce_sample(z, u, top_k=torch.full((n,), 50, dtype=torch.int32, device="cuda"))
    assert tok.tolist() == [head.sample(f64(z)[i], float(u[i]), 1.0, 50, 1.0, 0.0)[0]
                            for i in range(n)]
