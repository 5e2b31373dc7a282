"""Microscaled quantisation and its inverse: bit for bit the FP64 reference's
codes and scales (a division by a power of two is exact, so there is one right
answer)."""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from head_testutil import DT, f64, rand
from oracle import head

pytestmark = pytest.mark.gpu
FMTS = ["e4m3", "e2m1"]


def check(x, fmt):
    q, s = vce.mx_quantize(x, fmt)
    rq, rs = head.quantize(f64(x), fmt)
    assert np.array_equal(s.cpu().numpy(), rs), "scales"
    assert np.array_equal(q.cpu().numpy(), head.pack(rq, fmt)), "codes"
    ref = head.dequantize(head.pack(rq, fmt), rs, fmt)
    for dt in (torch.bfloat16, torch.float32):
        v = vce.mx_dequantize(q, s, fmt, dt)
        want = torch.from_numpy(ref).to(dt)
        assert torch.equal(torch.nan_to_num(v.cpu(), nan=-12345.0),
                           torch.nan_to_num(want, nan=-12345.0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (1, 2304), (257, 96), (33, 4096),
                                    (5, 8160)])
def test_quantize(rows, K, dtype, fmt):
    x = rand((rows, K), dtype, rows + K)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), device="cuda").float()).to(x.dtype)
    check(x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_every_bf16_value(fmt):
    """All 65536 bit patterns, each behind a largest value that puts the whole
    grid, its ties and its denormals within reach, and blocks of neighbours."""
    allv = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    neighbours = allv.view(-1, 32)
    check(neighbours.cuda(), fmt)
    spread = allv.view(32, 2048).t().contiguous()
    check(spread.cuda(), fmt)
    near = allv[(allv.float().abs() <= 448) & (allv.float().abs() >= 2.0 ** -12)]
    near = near[:near.numel() // 31 * 31].view(-1, 31)
    top = torch.full((near.shape[0], 1), 448.0, dtype=torch.bfloat16)
    check(torch.cat([top, near], 1).cuda(), fmt)
    check(torch.cat([near * (6.0 / 448), top * (6.0 / 448)], 1).to(torch.bfloat16).cuda(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_edges_fp32(fmt):
    """Largest values on both sides of a scale's limit, denormals, zeros of both
    signs, the ends of FP32, NaN and infinities."""
    rows = []
    vm = head.vmax(fmt)
    for e in (-140, -130, -127, -126, -100, -1, 0, 1, 100, 117, 119, 120):
        for m in (vm, np.nextafter(np.float32(vm), np.float32(1e9)),
                  np.nextafter(np.float32(vm), np.float32(0)), vm / 2, 1.0):
            with np.errstate(over="ignore", under="ignore"):
                top = np.float32(np.float64(m) * 2.0 ** e)
            if not np.isfinite(top):
                continue
            r = np.linspace(-1, 1, 32).astype(np.float32) * top
            r[7] = top
            rows.append(r)
    z = np.zeros(32, np.float32)
    rows += [z, -z, np.full(32, np.finfo(np.float32).max, np.float32),
             np.full(32, 1e-45, np.float32)]
    for bad in (np.nan, np.inf, -np.inf):
        r = np.linspace(-3, 3, 32).astype(np.float32)
        r[31] = bad
        rows.append(r)
    check(torch.from_numpy(np.stack(rows)).cuda(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_strides(dtype, fmt):
    big = rand((40, 135), dtype, 3)
    for x in (big[:, 3:67], big[::2, :64], big[5:6].expand(9, 135)[:, :96], big[1:, 7:39],
              rand((7, 3, 64), dtype, 4)[:, 1]):
        check(x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize_every_code_and_scale(fmt):
    codes = np.arange(256, dtype=np.uint8)
    q = np.tile(codes if fmt == "e4m3" else codes, (256, 1))
    K = 256 if fmt == "e4m3" else 512
    s = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, K // 32))
    ref = head.dequantize(q, s, fmt)
    for dt in (torch.float32, torch.bfloat16):
        v = vce.mx_dequantize(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), fmt, dt)
        want = torch.from_numpy(ref).to(dt)
        assert torch.equal(torch.nan_to_num(v.cpu(), nan=-12345.0, posinf=1, neginf=-1),
                           torch.nan_to_num(want, nan=-12345.0, posinf=1, neginf=-1))


def test_empty_and_neighbours():
    for fmt in FMTS:
        q, s = vce.mx_quantize(torch.empty((0, 64), device="cuda"), fmt)
        assert q.shape[0] == 0 and s.shape == (0, 2)
        assert vce.mx_dequantize(q, s, fmt).shape == (0, 64)
    x = rand((3, 96), "bf16", 5)
    q = torch.full((5, 96), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((5, 3), 9, dtype=torch.uint8, device="cuda")
    vce.mx_quantize(x, "e4m3", out=(q[1:4].view(3, 96), s[1:4]))
    assert (q[0] == 9).all() and (q[4] == 9).all() and (s[0] == 9).all() and (s[4] == 9).all()


def test_graph():
    x = rand((50, 2304), "bf16", 6)
    g = torch.cuda.CUDAGraph()
    vce.mx_quantize(x, "e2m1")
    with torch.cuda.graph(g):
        q, s = vce.mx_quantize(x, "e2m1")
        v = vce.mx_dequantize(q, s, "e2m1")
    for k in range(4):
        x.copy_(rand((50, 2304), "bf16", 7 + k))
        g.replay()
        eq, es = vce.mx_quantize(x, "e2m1")
        ev = vce.mx_dequantize(eq, es, "e2m1")
        torch.cuda.synchronize()
        assert torch.equal(q, eq) and torch.equal(s, es) and torch.equal(v, ev)
