"""The row by row check of ple_kv_attention's tests finds what a wrong swizzle, remainder or join would leave
behind. No GPU: the mistakes are planted in the float64 result."""

import numpy as np
import pytest

from _four_bit import Batch, bits
from _rows import faults, reference
from oracle.numerics import bf16_bits_to_f64, f64_to_bf16_bits

CASES = [([70, 1, 33], [70, 30, 150], 8, 2, 128), ([4, 1, 0, 9], [70, 1, 5, 133], 8, 1, 64), ([30, 2], [90, 40], 2, 1, 256)]


@pytest.fixture(scope="module", params=range(len(CASES)))
def case(request):
    queries, lens, heads, kv_heads, dim = CASES[request.param]
    b = Batch(queries, lens, heads, kv_heads, dim, 16, seed=request.param)
    ref = reference(b, bits(b.rows(heads)))
    return bf16_bits_to_f64(f64_to_bf16_bits(ref[0])), ref


def test_the_rounded_result_passes(case):
    got, ref = case
    assert faults(got, *ref) == []


@pytest.mark.parametrize("mistake", ["eight zeros", "another head's quarter", "a sign", "a neighbour's row", "a lost position",
                                     "values in bf16"])
def test_mistakes_are_found(case, mistake):
    got, ref = case
    got = got.copy()
    T, H, D = got.shape
    if mistake == "eight zeros":
        got[T // 2, 1, 8:16] = 0.0
    elif mistake == "another head's quarter":
        got[T - 1, 0, D // 4:D // 2] = got[T - 1, 1, D // 4:D // 2]
    elif mistake == "a sign":
        got[T - 1, :, 5] *= -1.0
    elif mistake == "a neighbour's row":
        got[T - 1, 1] = got[T - 2, 1]
    elif mistake == "a lost position":
        got[T - 1] *= 1.02
    else:  # another rounding of 2^-8 everywhere
        rng = np.random.default_rng(0)
        got = bf16_bits_to_f64(f64_to_bf16_bits(ref[0] * (1 + rng.uniform(-1, 1, got.shape) * 2.0 ** -8)))
        if got.size < 1000:
            return
    assert faults(got, *ref) != []
