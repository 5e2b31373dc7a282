"""ce_sample where a row's candidates fill the room that LDS has for them (4096), just fit it or
just do not: short rows kept almost whole, and top-k between half of it and all of it, whose
candidates lie spread over many groups of 32 tokens."""
import numpy as np
import pytest
import torch

from test_parity_sample import INF, normal, run

pytestmark = pytest.mark.gpu


def uniform(N, seed):
    return np.random.default_rng(seed).random(N, dtype=np.float32).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [3900, 3969, 4033, 4095, 4096])
def test_short_rows_kept_whole(V, dtype):
    """Groups and candidates together pass 4096, the candidates alone do not."""
    N = 600
    z = normal(N, V, dtype, V)
    u = uniform(N, V)
    run(z, u, p=[0.99999] * N, T=[4.0] * N)
    run(z, u, k=[V - 1 - i % 40 for i in range(N)])
    run(z, u, mp=[1e-12] * N, T=[2.0] * N)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V,live", [(9000, 4100), (20011, 4096), (32000, 3000), (200003, 4000)])
def test_large_top_k_that_fits(V, live, dtype):
    """Top-k of 2100 to 4096 with `live` tokens above a mask at random places."""
    N = 40
    z = normal(N, V, dtype, V)
    g = torch.Generator().manual_seed(V + 1)
    keep = torch.rand((N, V), generator=g).argsort(1)[:, :live].cuda()
    masked = torch.full_like(z, -INF)
    masked.scatter_(1, keep, z.gather(1, keep))
    u = uniform(N, live)
    k = [int(v) for v in np.linspace(2100, 4096, N)]
    run(z, u, k=k)
    run(masked, u, k=k)
    run(masked, u, k=k, p=[0.9, 0.999] * (N // 2), T=[1.0, 3.0] * (N // 2))
