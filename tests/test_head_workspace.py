"""What ce_sample asks for as workspace, and that it stays within it."""
import pytest
import torch

import vocabulary_cross_entropy_amd as vce
from vocabulary_cross_entropy_amd import binding


def test_short_rows_need_no_histogram():
    """Rows that are served whole (up to 4096 tokens) need their 256 group maxima and one of the
    segment; longer ones 16 KB of histogram each besides."""
    size = binding.lib().ce_sample_workspace_size
    for N in (1, 3, 1000, 1 << 20):
        for V in (1, 1000, 4096):
            assert N * 1028 <= size(N, V) <= N * 1028 + 1024
        assert size(N, 4097) >= N * (1028 + 16384)
    assert size(1 << 20, 1000) < 2 << 30


@pytest.mark.gpu
@pytest.mark.parametrize("V", [7, 4096, 4097, 9000])
@pytest.mark.parametrize("N", [1, 5, 300])
def test_no_byte_beyond(N, V):
    n = vce.ce_sample_workspace_size(N, V)
    buf = torch.full((n + 512,), 170, dtype=torch.uint8, device="cuda")
    z = torch.randn((N, V), device="cuda")
    u, p = torch.rand(N, device="cuda"), torch.full((N,), 0.999, device="cuda")
    k = torch.full((N,), V // 2, dtype=torch.int32, device="cuda")
    for args in ((), (None, k), (None, None, p), (None, k, p)):
        buf.fill_(170)
        got = vce.ce_sample(z, u, *args, workspace=buf[:n])
        assert torch.equal(got, vce.ce_sample(z, u, *args))
        assert (buf[n:] == 170).all()
