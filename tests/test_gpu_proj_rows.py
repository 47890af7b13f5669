"""ple_proj_w4 on the GPU against float64, with the bound of what the kernels do. Codes less zero points, over 64,
are exact in bf16 and so are their products with x in float32; what is rounded is float32 sums - two steps of a
tensor core's 16 columns with up to two units of 2^-24 each, one of 2^-24 for each group's scale and for each part
that is joined, relative to the sum of the absolute products - and the result, 2^-8 of it at most. A whole output's
error is its rounding, uniform within half a step of each element."""

import numpy as np
import pytest
import torch

from _four_bit import bits, oracle
from _helpers import bf16_values
from test_gpu_proj_w4 import project, weight

pytestmark = pytest.mark.gpu


def faults(got, want, total, E, group):
    err = np.abs(got - want)
    single = (4 * group / 16 + E / group + 12) * 2.0 ** -24 * total
    found = []
    if not (err <= 2.0 ** -8 * np.abs(want) + single).all():
        found.append(f"an element: {(err - 2.0 ** -8 * np.abs(want) - single).max():.3g} above its bound")
    step = 2.0 ** (np.floor(np.log2(np.abs(np.where(want != 0, want, 1.0)))) - 7)
    limit = 1.15 * np.sqrt((step ** 2).sum() / 12 + (single ** 2).sum())
    if np.sqrt((err ** 2).sum()) > limit:
        found.append(f"the whole: {np.sqrt((err ** 2).sum()):.4g}, bound {limit:.4g}")
    return found


# both kernels, every number of token tiles, columns that end inside a block, columns shared out or not
@pytest.mark.parametrize("T,N,E,group", [(1, 2000, 4096, 128), (8, 300, 1056, 32), (16, 700, 832, 64), (30, 600, 2176, 128),
                                         (24, 4870, 320, 64), (33, 700, 4096, 128), (64, 2500, 832, 64), (64, 20001, 352, 32),
                                         (129, 500, 1152, 128)])
@pytest.mark.parametrize("with_zeros", [False, True])
def test_against_float64(T, N, E, group, with_zeros):
    codes, scales, zeros = weight(N, E, group, with_zeros, seed=N + E)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    out = project(x.cuda(), codes, scales, zeros)
    got = faults(bf16_values(bits(out)), *oracle.proj_w4(bits(x), codes, bits(scales), zeros, group), E, group)
    assert not got, got


@pytest.mark.parametrize("T", [1, 12, 40])
def test_zero_points_of_any_byte_and_large_inputs(T):
    """Zero points up to 255 make (c - z) of eight bits, which bf16 still holds."""
    codes, scales, _ = weight(333, 1024, 64, True, seed=T)
    zeros = np.random.default_rng(T).integers(0, 256, (333, 16)).astype(np.uint8)
    x = (torch.randn(T, 1024, generator=torch.Generator().manual_seed(T)) * 2.0 ** 60 + 2.0 ** 62).to(torch.bfloat16)
    out = project(x.cuda(), codes, scales, zeros)
    got = faults(bf16_values(bits(out)), *oracle.proj_w4(bits(x), codes, bits(scales), zeros, 64), 1024, 64)
    assert not got, got


@pytest.mark.parametrize("T,N", [(1, 600), (12, 600), (40, 600), (64, 40000)])
def test_scales_near_the_largest(T, N):
    """Scales of 2^122 to 2^127 on inputs small enough for a finite result, and on zeros."""
    E, group = 512, 128
    codes, scales, zeros = weight(N, E, group, True, seed=T)
    scales = (scales.float() / 0.02 * 2.0 ** 127).to(torch.bfloat16)
    x = (torch.randn(T, E, generator=torch.Generator().manual_seed(T)) * 2.0 ** -20).to(torch.bfloat16)
    x[T // 2:, :] = 0.0 if T > 1 else x[0]
    out = project(x.cuda(), codes, scales, zeros)
    want, total = oracle.proj_w4(bits(x), codes, bits(scales), zeros, group)
    got = faults(bf16_values(bits(out)), want, total, E, group)
    assert not got, got
