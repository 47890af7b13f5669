"""pack_mx8 of weights in any order of memory (no GPU)."""

import pytest
import torch

from hashed_gram_embedding_gb300 import pack_mx8


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("view", ["transposed", "columns", "every other"])
def test_codes_lie_row_by_row(view, dtype):
    g = torch.Generator().manual_seed(0)
    w = torch.randn(256, 512, generator=g).to(dtype)
    w = {"transposed": w.t(), "columns": w[:, 128:384], "every other": w[::2, ::2]}[view]
    codes, scales = pack_mx8(w)
    want = pack_mx8(w.contiguous())
    assert codes.is_contiguous() and scales.is_contiguous()
    assert codes.shape == w.shape and torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_a_parameter():
    codes, scales = pack_mx8(torch.nn.Parameter(torch.ones(4, 128)))
    assert not codes.requires_grad and not scales.requires_grad
