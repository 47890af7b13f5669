"""What the 8-bit step's Python calls refuse before the library is asked (no GPU)."""

from types import SimpleNamespace

import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from hashed_gram_embedding_gb300 import _lib, build


def codes_and_scales(rows, columns):
    """Stands in for tensors too large to make."""
    def like(*shape):
        return SimpleNamespace(dtype=torch.uint8, is_contiguous=lambda: True, is_cuda=True, shape=shape,
                               numel=lambda: shape[-1])
    return like(rows, columns), like(-(-rows // 128) * columns * 4)


def test_weights_that_no_product_takes():
    """Refused where a block is built, not in its first step."""
    w1, w2 = ple.pack_mx8(torch.zeros(256, 128)), ple.pack_mx8(torch.zeros(128, 128))
    with pytest.raises(ValueError, match="w_gate_up"):
        ple.PLEFeedForward(w1, w2, None, 4)  # on the host
