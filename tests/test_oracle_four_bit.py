"""The 4-bit step's oracle pinned to things other than itself: torch's own
operations on the CPU, closed forms, hand values."""

import numpy as np
import torch

from _four_bit import Batch, bits, oracle, rotation_table
from oracle.numerics import bf16_bits_to_f64


def test_quantise_hand_values():
    # 0 .. 15 in steps of 1: scale 1 (15 * fl(1/15) rounds to 1 in bf16), offset 0, codes themselves
    codes, pair = oracle.quantise(np.arange(16, dtype=np.float32))
    assert codes.tolist() == list(range(16)) and bf16_bits_to_f64(pair).tolist() == [1.0, 0.0]
    # ties go to the even code; below the offset's rounding and above the last code are clamped
    codes, pair = oracle.quantise(np.array([-2, -1.5, -0.5, 13], np.float32))
    assert codes.tolist() == [0, 0, 2, 15] and bf16_bits_to_f64(pair).tolist() == [1.0, -2.0]
    assert oracle.quantise(np.full(4, 5.0, np.float32))[0].tolist() == [0, 0, 0, 0]


def test_quantised_rows_are_within_half_a_step():
    x = np.random.default_rng(0).normal(0, 2, (200, 64)).astype(np.float32)
    for row in x:
        codes, pair = oracle.quantise(row)
        s, m = bf16_bits_to_f64(pair)
        # half a step, plus the rounding of the offset and of 15 scales
        assert np.abs(codes * s + m - row).max() <= s / 2 + 2 ** -8 * (abs(row.min()) + 15 * s)


def test_rotation_is_a_complex_product_and_keeps_the_rest():
    cs = rotation_table(50, 32)
    x = np.random.default_rng(1).normal(size=(3, 64)).astype(np.float32)
    for interleaved in (False, True):
        y = oracle.rotate(x, cs, 37, interleaved)
        a = (x[:, 0:32:2], x[:, 1:32:2]) if interleaved else (x[:, :16], x[:, 16:32])
        b = (y[:, 0:32:2], y[:, 1:32:2]) if interleaved else (y[:, :16], y[:, 16:32])
        turn = np.exp(1j * 37 * 10000.0 ** (-np.arange(0, 32, 2) / 32))
        assert np.allclose((a[0] + 1j * a[1]) * turn, b[0] + 1j * b[1], atol=2e-6)
        assert np.array_equal(x[:, 32:], y[:, 32:])


def test_append_then_read_and_nothing_else_changes():
    b = Batch([2, 0, 3], [2, 5, 20], 4, 2, 64, 16, seed=2)
    before = b.cache.copy()
    q, k, v = b.rows(4), b.rows(2), b.rows(2)
    out = oracle.append(bits(q), bits(k), bits(v), None, b.cache, b.table, b.qsl, b.lens)
    assert np.array_equal(out, bits(q))
    for t, r, p in oracle.tokens(b.qsl, b.lens, b.T):
        got = oracle.read(b.cache, b.table, r, p, 64)
        for i, x in enumerate((k, v)):
            x = x[t].float().numpy()
            step = (x.max(-1) - x.min(-1))[:, None] / 15
            assert (np.abs(got[i] - x) <= step / 2 + 2 ** -8 * (np.abs(x.min(-1))[:, None] + 15 * step)).all()
            page, sub, slot = oracle.place(b.cache, b.table, r, p)
            for h in range(2):
                for now, was in zip(oracle.block_parts(b.cache[page, h, sub], 64),
                                    oracle.block_parts(before[page, h, sub], 64)):
                    was[slot] = now[slot]
    assert np.array_equal(b.cache, before)


def test_attention_matches_torch_on_the_read_values():
    for causal, window in ((True, 0), (True, 5), (False, 0)):
        b = Batch([3, 9, 1], [3, 30, 17], 6, 2, 64, 16, seed=3)
        q = b.rows(6)
        got = oracle.attention(bits(q), b.cache, b.table, b.qsl, b.lens, 0.125, causal, window)[0]
        for r in range(3):
            n, L = b.queries[r], int(b.lens[r])
            kv = torch.from_numpy(np.stack([oracle.read(b.cache, b.table, r, p, 64) for p in range(L)]))
            mask = torch.ones(n, L, dtype=torch.bool)
            if causal:
                mask = mask.tril(L - n)
                if window:
                    mask &= mask.new_ones(n, L).triu(L - n - window + 1)
            k, v = kv[:, 0].transpose(0, 1), kv[:, 1].transpose(0, 1)
            k, v = k.repeat_interleave(3, 0), v.repeat_interleave(3, 0)
            rows = slice(b.qsl[r], b.qsl[r + 1])
            want = torch.nn.functional.scaled_dot_product_attention(
                q[rows].double().transpose(0, 1), k, v, attn_mask=mask, scale=0.125).transpose(0, 1)
            assert np.allclose(got[rows], want.numpy(), atol=1e-12)


def test_projection_matches_a_dense_product():
    rng = np.random.default_rng(4)
    codes = rng.integers(0, 256, (5, 32), dtype=np.uint8)
    scales = torch.from_numpy(rng.uniform(0.01, 0.1, (5, 2)).astype(np.float32)).to(torch.bfloat16)
    zeros = rng.integers(0, 16, (5, 2)).astype(np.uint8)
    x = torch.from_numpy(rng.normal(size=(3, 64)).astype(np.float32)).to(torch.bfloat16)
    for z in (zeros, None):
        got, total = oracle.proj_w4(bits(x), codes, bits(scales), z, 32)
        for n in range(5):
            for t in range(3):
                terms = [float(x[t, e]) * float(scales[n, e // 32]) *
                         ((int(codes[n, e // 2]) >> (4 * (e % 2)) & 15) - (8 if z is None else int(z[n, e // 32])))
                         for e in range(64)]
                assert abs(got[t, n] - sum(terms)) < 1e-12 and abs(total[t, n] - sum(map(abs, terms))) < 1e-12
