"""Calls of the adapted head's operators that the documentation allows and the other tests do not make:
single outputs, broadcast inputs, the same tensor twice, one workspace for two graphs."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import U, f64, rand
from oracle import beam
from vocabulary_cross_entropy_amd import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V", [(5, 40), (300, 4352), (300, 4353)])
def test_each_gradient_alone(M, V, dtype):
    """Any subset of dx, da and db has the bits that all three have together."""
    H, n, r = 72, 3, 16
    x, w = rand((M, H), "bf16", 1), rand((V, H), "bf16", 2, 0.1)
    a, b = rand((n, r, H), "bf16", 3, 0.1), rand((n, V, r), "bf16", 4, 0.1)
    dy = rand((M, V), "fp32", 5, 0.1).to(dtype)
    k = (torch.arange(M, device="cuda") % (n + 1) - 1).to(torch.int32)
    ws = vce.lora_backward_workspace(M, H, V, n, r, dtype)
    code = binding.DTYPE_BF16 if dtype == torch.bfloat16 else binding.DTYPE_FP32
    shapes = (((M, H), torch.bfloat16), ((n, r, H), torch.float32), ((n, V, r), torch.float32))

    def call(wanted, weight):
        out = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in shapes]
        at = [o.data_ptr() if u else None for o, u in zip(out, wanted)]
        rc = binding.lib().lora_backward(
            dy.data_ptr(), code, V, x.data_ptr(), H, M, H, V, a.data_ptr(), b.data_ptr(), n, r,
            k.data_ptr(), None, weight.data_ptr() if weight is not None else None, None, *at,
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        return out

    for weight in (w, None):
        full = call((1, 1, 1), weight)
        for wanted in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (1, 0, 1), (0, 1, 1)):
            for got, ref, u in zip(call(wanted, weight), full, wanted):
                assert torch.equal(got, ref if u else torch.full_like(ref, 7.0)), wanted


def test_beams_of_one_row():
    """Logits broadcast over the beams and over the requests (strides of zero)."""
    z = torch.randn(1001, device="cuda") * 3
    s = -torch.rand((3, 4), device="cuda")
    score, par, tok = vce.beam_step(z.expand(3, 4, 1001), s, 9)
    for b in range(3):
        v, p, t = beam.step(np.tile(f64(z), (4, 1)), f64(s)[b], 9)
        assert par[b].tolist() == p.tolist() and tok[b].tolist() == t.tolist()
        assert (np.abs(f64(score)[b] - v) <= U * np.abs(v) + 2e-11).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_one_gradient_for_two_parameters(bits):
    g = torch.randn(500, device="cuda")
    p = [torch.randn(500, device="cuda") for _ in range(2)]
    q = [t.clone() for t in p]
    st, su = vce.adamw_state(p, bits), [vce.adamw_state([t], bits) for t in q]
    vce.adamw_step(p, [g, g], st, 1e-2, 1)
    for t, s in zip(q, su):
        vce.adamw_step([t], [g], s, 1e-2, 1)
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    norm, _ = vce.grad_norm([g, g])
    want = np.sqrt(2 * (f64(g) ** 2).sum())
    assert abs(norm.item() - want) <= 2 * U * want


@pytest.mark.parametrize("count", [64, 65, 200])
def test_more_tensors_than_a_launch_takes(count):
    """Tables of 64: each tensor as in a call of its own, and the norm over all."""
    sizes = [1 + 37 * i % 700 for i in range(count)]
    p = [torch.randn(n, device="cuda") for n in sizes]
    g = [torch.randn(n, device="cuda") for n in sizes]
    q = [t.clone() for t in p]
    vce.adamw_step(p, g, vce.adamw_state(p), 1e-2, 1)
    for i in sorted({0, 62, 63, count - 1}):
        vce.adamw_step([q[i]], [g[i]], vce.adamw_state([q[i]]), 1e-2, 1)
        assert torch.equal(p[i], q[i]), i
    want = np.sqrt(sum((f64(t) ** 2).sum() for t in g))
    assert abs(vce.grad_norm(g)[0].item() - want) <= 2 * U * want


def test_two_graphs_and_one_workspace():
    """Two captured calls of different sizes that take turns on one workspace."""
    H, V, n, r = 64, 2000, 4, 8
    a, b = rand((n, r, H), "bf16", 1), rand((n, V, r), "bf16", 2)
    w = rand((V, H), "bf16", 3, 0.1)
    calls = []
    ws = vce.lora_backward_workspace(700, H, V, n, r)
    for i, M in enumerate((9, 700)):
        x, dy = rand((M, H), "bf16", 4 + i), rand((M, V), "bf16", 6 + i, 0.1)
        k = (torch.arange(M, device="cuda") % (n + 1) - 1).to(torch.int32)
        out = [torch.empty((M, V), dtype=torch.bfloat16, device="cuda")]
        out += [torch.empty((M, H), dtype=torch.bfloat16, device="cuda"),
                torch.empty((n, r, H), device="cuda"), torch.empty((n, V, r), device="cuda")]

        def run(x=x, dy=dy, k=k, out=out):
            vce.lora_forward(x, a, b, k, w, out=out[0], workspace=ws)
            vce.lora_backward(dy, x, a, b, k, w, out=out[1:], workspace=ws)
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        calls.append((graph, out, [t.clone() for t in out], run))  # run holds the inputs
    for _ in range(4):
        for graph, out, *_ in calls:
            for t in out:
                t.fill_(3.0)
            ws.fill_(255)
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in calls:
            assert all(torch.equal(t, u) for t, u in zip(out, want))


def test_reorder_twice_with_one_parent():
    """Two calls in a row, and one state given as two halves of one array."""
    t = torch.randn((3, 4, 2, 50), device="cuda")
    ref = t.clone()
    par = torch.tensor([[1, 0, 3, 3], [0, 1, 2, 3], [3, 3, 3, -1]], dtype=torch.int32, device="cuda")
    idx = torch.where(par < 0, torch.arange(4, device="cuda"), par.long())
    for _ in range(2):
        vce.beam_reorder([t[:, :, 0], t[:, :, 1]], par)
        ref = torch.stack([ref[i][idx[i]] for i in range(3)])
    assert torch.equal(t, ref)
