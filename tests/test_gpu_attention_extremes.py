"""ple_kv_attention on the GPU where values, keys and queries lie far from one: what float32 holds of the
float64 result, row by row (the bounds are those of _rows.py)."""

import numpy as np
import pytest
import torch

from _four_bit import Batch, bits
from _helpers import bf16_values, dev_err_word
from _rows import F16, U, faults, reference
from test_gpu_kv_attention import attend

pytestmark = pytest.mark.gpu


def run(b, q, scale=None, weights=F16, **kw):
    err = dev_err_word()
    out = attend(b, q, scale=scale, err=err, **kw)
    assert int(err.item()) == 0
    got = faults(bf16_values(bits(out)), *reference(b, bits(q), scale), weights=weights)
    assert not got, got


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries,length", [(120, 256), (40, 2600), (3, 300)])
@pytest.mark.parametrize("first,then", [(1e-12, 1e30), (1e30, 1e-12), (1e-6, 1e4), (1e-25, 1e25)])
def test_values_that_leap(dim, queries, length, first, then):
    """Values of one size for half of the positions, of another for the rest: the sum of the weights outlives
    what the outputs are scaled by."""
    b = Batch([queries], [length], 4, 1, dim, 16, seed=3, k_mean=0.0)
    for p in range(length):
        b.put(0, p, b.rng.normal(0, 1, (1, dim)), b.rng.normal(0, first if p < length // 2 else then, (1, dim)))
    run(b, b.rows(4), weights=U if queries == 3 else F16)


@pytest.mark.parametrize("queries,length", [(60, 2600), (300, 1500)])
@pytest.mark.parametrize("at", [0, 700, 1300])
def test_one_huge_value_among_many_small_weights(queries, length, at):
    """A value of 2e36 takes a weight 2^12 times those of the others, which together weigh as much."""
    b = Batch([queries], [length], 4, 1, 128, 16, seed=5)
    for p in range(length):
        b.put(0, p, np.zeros((1, 128)), b.rng.normal(0, 1, (1, 128)))
    b.put(0, at, np.full((1, 128), 0.55), b.rng.uniform(0.5, 1, (1, 128)) * 2e36)
    q = b.rows(4)
    q[:] = q.abs() + 0.5
    run(b, q)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", [2, 100])
@pytest.mark.parametrize("exponent", [-115, 95, 104, 122])
def test_queries_of_any_size(dim, queries, exponent):
    """Every kernel takes the queries that the others take: rows near both ends of bf16's range, keys to match."""
    b = Batch([queries], [150], 4, 1, dim, 16, seed=7, k_mean=0.0)
    for p in range(150):
        b.put(0, p, b.rng.normal(0, 2.0 ** min(-exponent, 100), (1, dim)), b.rng.normal(0, 1, (1, dim)))
    q = b.rows(4, 2.0 ** exponent)
    q[0, 1] = 0.0
    run(b, q)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("queries", [2, 100])
def test_small_elements_of_a_query_count(dim, queries):
    """One element of a query row 2^12 times the others, met by zeros in the keys."""
    b = Batch([queries], [150], 4, 1, dim, 16, seed=9)
    for p in range(150):
        k = np.abs(b.rng.normal(0, 1, (1, dim)))
        k[:, 3] = 0.0
        b.put(0, p, k, b.rng.normal(0, 1, (1, dim)))
    q = b.rows(4)
    q[:, :, 3] = 4096.0
    run(b, q)
