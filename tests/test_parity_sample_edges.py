"""ce_sample at the ends of what temperatures and logits may be."""
import numpy as np
import pytest
import torch

from head_testutil import DT
from test_parity_sample import FMAX, normal, run

pytestmark = pytest.mark.gpu


def uniform(N, seed):
    return np.random.default_rng(seed).random(N, dtype=np.float32).tolist()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [300, 4096, 5000, 40000])
def test_min_p_where_every_weight_is_one(V, dtype):
    """T so large that each weight is 1 in FP64: min_p = 1 keeps every token, alone as after
    the other filters."""
    N = 24
    z, u = normal(N, V, dtype, V), uniform(N, V)
    T = [1e20, 1e30] * (N // 2)
    run(z, u, T=T, mp=[1.0] * N)
    run(z, u, T=T, mp=[2.0] * N, k=[V // 2] * N)
    run(z, u, T=T, mp=[1.0] * N, p=[0.7] * N)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,V", [(8, 300), (8, 6000), (300, 9000)])
def test_distances_beyond_fp32(N, V, dtype):
    """Logits over all of FP32 under a temperature to match: a token whose distance from the
    maximum overflows FP32 weighs what the formula says, and min-p's bound may overflow too."""
    g = torch.Generator().manual_seed(V)
    z = ((torch.rand((N, V), generator=g) * 2 - 1) * (0.99 * FMAX)).to(DT[dtype]).cuda()
    u, T = uniform(N, V + 1), [3e38] * N
    run(z, u, T=T)
    run(z, u, T=T, mp=[0.11 + 0.05 * (i % 8) for i in range(N)])
    run(z, u, T=T, mp=[0.2] * N, p=[0.9] * N)
    run(z, u, T=T, k=[40, V - 1] * (N // 2))
    run(z, u, T=T, p=[0.5, 0.97] * (N // 2))
