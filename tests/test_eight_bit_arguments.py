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


@pytest.mark.parametrize("rows,columns", [(1, 2**31), (1, 2**32 + 128), (3, 2**33 + 256)])
def test_columns_past_32_bits(rows, columns):
    """They would reach the library as what is left of them in 32 bits."""
    with pytest.raises(ValueError, match="codes"):
        _lib._mx8("codes, scales", *codes_and_scales(rows, columns))
    assert _lib._mx8("codes, scales", *codes_and_scales(rows, 2**31 - 128)) == (rows, 2**31 - 128)


def test_scale_bytes_of_sizes_past_32_bits():
    build.build()
    assert ple.ple_mx8_scale_bytes(1, 2**32 + 128) == 0 and ple.ple_mx8_scale_bytes(1, -2**32 + 128) == 0
    assert ple.ple_mx8_scale_bytes(2**64 + 1, 128) == 0
    assert ple.ple_mx8_scale_bytes(130, 256) == 2048
