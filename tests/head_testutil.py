"""Helpers of the tests of the operators around the head.

Bounds count roundings: u = 2^-24 for an FP32 operation, and half a step of
the stored type (2^-8 of the value for BF16, 2^-24 for FP32) for the result.
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -126  # below the normal range a rounding is absolute
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def assert_within(got, ref, bound, what):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, f"{what}: {got.shape} against {ref.shape}"
    bad = ~(np.abs(got - ref) <= bound)
    same_nan = np.isnan(got) & np.isnan(ref)
    same_inf = np.isinf(ref) & (got == ref)
    bad &= ~(same_nan | same_inf)
    if bad.any():
        i = np.unravel_index(np.argmax(bad), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside, first at {i}: "
                             f"{got[i]!r} against {ref[i]!r}")
