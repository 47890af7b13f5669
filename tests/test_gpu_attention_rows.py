"""ple_kv_attention on the GPU against float64, row by row and sixteen elements at a time: the bounds of
_rows.py, which are those of f16 weights, values and keys and one rounding of the result."""

import pytest
import torch

from hashed_gram_embedding_gb300 import _lib

from _four_bit import Batch, bits
from _helpers import bf16_values, dev_err_word
from _rows import faults, reference
from test_gpu_kv_attention import LAYOUTS, attend

pytestmark = pytest.mark.gpu


def run(b, causal=True, window=0, scale=None, **kw):
    q = b.rows(b.heads)
    err = dev_err_word()
    out = attend(b, q, causal, window, scale=scale, err=err, **kw)
    assert int(err.item()) == 0
    got = faults(bf16_values(bits(out)), *reference(b, bits(q), scale, causal, window))
    assert not got, got


@pytest.mark.parametrize("heads,kv_heads,dim", LAYOUTS)
@pytest.mark.parametrize("page", [16, 48])
def test_single_tokens(heads, kv_heads, dim, page):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200, 0, 410]
    run(Batch([1] * len(lens), lens, heads, kv_heads, dim, page, seed=dim + heads), hint=1)


@pytest.mark.parametrize("heads,kv_heads,dim", LAYOUTS)
@pytest.mark.parametrize("hint", [0, 9])
def test_few_tokens(heads, kv_heads, dim, hint):
    run(Batch([4, 1, 0, 9, 2, 3], [70, 1, 5, 9, 133, 340], heads, kv_heads, dim, 16, seed=7, pad=3), hint=hint)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 2, 128), (5, 1, 128), (2, 1, 256), (16, 1, 256)])
@pytest.mark.parametrize("page", [16, 80])
def test_prefill_chunks(heads, kv_heads, dim, page):
    run(Batch([97, 1, 130, 3, 64], [97, 30, 300, 3, 191], heads, kv_heads, dim, page, seed=page), hint=130)


@pytest.mark.parametrize("queries,lens", [([1, 3], [2777, 900]), ([40, 2], [2500, 700])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_contexts(queries, lens, dim):
    run(Batch(queries, lens, 4, 1, dim, 32, seed=11))


@pytest.mark.parametrize("queries,lens", [([1, 4, 40], [50, 300, 140]), ([150], [260])])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 33), (True, 100), (False, 0)])
def test_masks(queries, lens, causal, window):
    run(Batch(queries, lens, 8, 2, 128, 16, seed=13), causal=causal, window=window)


@pytest.mark.parametrize("queries,lens", [([1, 3], [150, 40]), ([100], [150])])
def test_keys_far_from_zero_and_large_scores(queries, lens):
    run(Batch(queries, lens, 8, 2, 128, 16, seed=37, k_mean=30.0), scale=0.02)
    run(Batch(queries, lens, 8, 2, 128, 16, seed=38), scale=1.0)


@pytest.mark.parametrize("size", [0.02, 0.3, 40.0, 800.0])
@pytest.mark.parametrize("queries,lens", [([1, 3], [150, 40]), ([100], [150])])
def test_values_of_ordinary_sizes(size, queries, lens):
    """Their ranges lie within what f16 weights serve."""
    b = Batch(queries, lens, 8, 2, 128, 16, seed=61)
    for r, n in enumerate(lens):
        for p in range(n):
            b.put(r, p, b.rng.normal(0, 1, (2, 128)), b.rng.normal(0, size, (2, 128)))
    run(b)


@pytest.mark.parametrize("queries,lens", [([1, 4], [90, 40]), ([100, 3], [130, 30])])
def test_bytes_that_no_token_sees_change_no_bit(queries, lens):
    """Scales of every size, NaN and infinity among them, behind the last position."""
    outs = []
    for garbage in (0, 1, 2, 3):
        b = Batch(queries, lens, 8, 2, 64, 16, seed=67)
        q = b.rows(8)
        for r, n in enumerate(lens):
            for p in range(n, -(-n // 16) * 16):
                page, sub, slot = b.table[r, p // 16], 0, p % 16
                pairs = b.cache[page, :, sub, 16 * 64:].view("uint16").reshape(-1, 2, 16, 2)
                pairs[:, :, slot] = (0x0000, 0x7F80, 0x7000, 0x1000)[garbage]
        outs.append(attend(b, q).cpu().view(torch.int16))
    for other in outs[1:]:
        assert torch.equal(outs[0], other)


@pytest.mark.parametrize("queries,lens", [([1] * 5, [700, 3, 90, 1500, 1]), ([4, 2], [900, 40]), ([200, 1], [300, 60]),
                                          ([40], [2600])])
def test_in_place(queries, lens):
    """The result in q's own memory: the same bits."""
    b = Batch(queries, lens, 8, 2, 128, 16, seed=43, pad=2)
    q = b.rows(8)
    want = attend(b, q)
    cache, table, qsl, lens_d = b.device()
    ws = torch.zeros(_lib.ple_kv_attention_workspace(8, 2, 128), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        x = q.cuda()
        _lib.ple_kv_attention(x, cache, table, qsl, lens_d, x, ws)
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))
