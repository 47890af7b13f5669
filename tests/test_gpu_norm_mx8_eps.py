"""ple_norm_mx8 with an eps of any size."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from oracle import eight_bit as oracle

from _eight_bit import check_mx8, room
from _helpers import bits, bf16_values

pytestmark = pytest.mark.gpu

OFF = 2.0 ** -18  # of the float32 norm: a sum of squares (its error halved by the root) and 6 roundings


@pytest.mark.parametrize("c", [128, 640, 16384])
@pytest.mark.parametrize("size", [1e-30, 1.0, 3e17, 1e19, 3e38])
@pytest.mark.parametrize("eps", [1e-45, 1e-38, 1e-6, 1.0, 1e30, 3.4028234e38])
def test_eps(c, size, eps):
    x = torch.from_numpy(np.random.default_rng(c).uniform(0.25, 1, (5, c)) * size).to(torch.float32).to(torch.bfloat16)
    x[2] = 0
    codes, scales = room(5, c)
    ple.ple_norm_mx8(x.cuda(), None, codes, scales, eps=eps)
    _, n = oracle.norm(bf16_values(bits(x)).reshape(x.shape), None, None, float(np.float32(eps)))
    # a result below 2^-126 is rounded by half of float32's least, at most
    check_mx8(codes, scales, n, OFF * np.abs(n) + 2.0 ** -149, f"{eps}")
