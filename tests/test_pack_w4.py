"""pack_w4 of weights in any order of memory (no GPU)."""

import pytest
import torch

from hashed_gram_embedding_gb300 import pack_w4


@pytest.mark.parametrize("view", ["transposed", "columns", "every other"])
def test_codes_lie_row_by_row(view):
    w = torch.randn(256, 512, generator=torch.Generator().manual_seed(0))
    w = {"transposed": w.t(), "columns": w[:, 128:384], "every other": w[::2, ::2]}[view]
    got, want = pack_w4(w), pack_w4(w.contiguous())
    assert all(g.is_contiguous() and torch.equal(g, a) for g, a in zip(got, want))


def test_a_parameter():
    assert not any(a.requires_grad for a in pack_w4(torch.nn.Parameter(torch.randn(4, 128))))
