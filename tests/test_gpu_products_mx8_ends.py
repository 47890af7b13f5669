"""ple_proj_mx8 at the ends of its ranges: the most tokens, many rows, many columns."""

import pytest
import torch

import hashed_gram_embedding_gb300 as ple

from _helpers import dev_err_word
from _mx8_sums import exact_operands

pytestmark = pytest.mark.gpu

MOST = 4194240  # tokens


@pytest.mark.parametrize("t,e,n", [(MOST, 128, 130), (MOST, 256, 7), (1, 128, 30_000_000), (40, 128, 9_000_001),
                                   (200, 128, 3_000_001), (1, 1 << 22, 200), (300, 1 << 20, 130)])
def test_ends(t, e, n):
    """Sums of whole numbers of a unit, of a product's at most 225 of them: at 2^22
    columns the sums' standard deviation is 75 * 2^11 < 2^18, and 2^24 is 100 of
    those; so all partial sums are exact."""
    x8, x, w8, w = exact_operands(t, e, n, device="cuda")
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    err = dev_err_word()
    ple.ple_proj_mx8(*x8, *w8, out, dev_err=err)
    assert int(err.item()) == 0
    step = 1 << 19
    for a in range(0, t, step):
        for b in range(0, n, step):
            want = x[a:a + step] @ w[b:b + step].T
            assert torch.equal(out[a:a + step, b:b + step], want.float().to(torch.bfloat16)), (a, b)


def test_one_token_more():
    codes = torch.empty((MOST + 1, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((ple.ple_mx8_scale_bytes(MOST + 1, 128),), dtype=torch.uint8, device="cuda")
    _, _, w8, _ = exact_operands(1, 128, 128, device="cuda")
    with pytest.raises(ple.PleError, match="UNSUPPORTED"):
        ple.ple_proj_mx8(codes, scales, *w8, torch.empty((MOST + 1, 128), dtype=torch.bfloat16, device="cuda"))
