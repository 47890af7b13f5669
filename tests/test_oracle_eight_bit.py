"""The 8-bit step's oracle against things other than itself, and pack_mx8
against the oracle (no GPU)."""

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import pack_mx8
from oracle import eight_bit as oracle


def test_layout_by_hand():
    # 256 columns: two pieces a row block; rows 0, 1, 32 and 128, blocks 0, 3, 4 and 7
    assert [oracle.scale_at(r, 0, 256) for r in (0, 1, 32, 128)] == [0, 16, 4, 1024]
    assert [oracle.scale_at(0, j, 256) for j in (0, 3, 4, 7)] == [0, 3, 512, 515]
    byte = np.random.default_rng(0).integers(0, 256, (200, 12), dtype=np.uint8)
    laid = oracle.lay_out(byte, 384)
    assert laid.size == 2 * 3 * 512 and np.array_equal(oracle.pick(laid, 200, 384), byte)
    # as a reshape
    whole = np.zeros((256, 12), np.uint8)
    whole[:200] = byte
    assert np.array_equal(laid, whole.reshape(2, 4, 32, 3, 4).transpose(0, 3, 2, 1, 4).ravel())


@pytest.mark.parametrize("top,byte", [(448.0, 127), (448.0 * (1 + 2 ** -20), 128), (1.75, 119), (1.0, 119),
                                      (1.7500001, 120), (0.0, 0), (2.0 ** -127, 0), (448 * 2.0 ** -127, 0),
                                      (449 * 2.0 ** -127, 1), (3.4e38, 247), (np.inf, 255), (np.nan, 255)])
def test_scale_of_a_block(top, byte):
    x = np.zeros((1, 128))
    x[0, 5] = -top
    _, got = oracle.quantise(x)
    assert got[0, 0] == byte and (got[0, 1:] == 0).all()


def test_codes_round_to_nearest_even():
    # a block whose power is 1: e4m3's values stay, halves between go to the even code
    y = oracle._MAGNITUDES
    for a in range(126):
        x = np.zeros((1, 128))
        x[0, 0], x[0, 1] = 448.0, (y[a] + y[a + 1]) / 2
        x[0, 2], x[0, 3] = y[a], -y[a + 1]
        codes, byte = oracle.quantise(x)
        assert byte[0, 0] == 127
        assert codes[0, 1] == a + a % 2 and codes[0, 2] == a and codes[0, 3] == 128 + a + 1


def test_values_and_torch_agree():
    rng = np.random.default_rng(1)
    x = rng.normal(0, 1, (130, 256)) * 2.0 ** rng.integers(-30, 30, (130, 1))
    codes, byte = oracle.quantise(x)
    there = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.values(codes, byte), there * np.repeat(2.0 ** (byte - 127.0), 32, 1))
    # half a step, and no more
    step = np.repeat(2.0 ** (byte - 127.0), 32, 1)
    assert (np.abs(oracle.values(codes, byte) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()


@pytest.mark.parametrize("rows,columns", [(1, 128), (37, 384), (128, 128), (257, 256)])
def test_pack_mx8(rows, columns):
    rng = np.random.default_rng(rows)
    x = (rng.normal(0, 1, (rows, columns)) * 10.0 ** rng.integers(-38, 37, (rows, 1))).astype(np.float32)
    x[0, :32] = 0
    x[-1, 32:64] = [2.0 ** -149] * 32
    x[rows // 2, 70] = np.nan
    x[rows // 3, 100] = -np.inf
    codes, scales = pack_mx8(torch.from_numpy(x))
    want, byte = oracle.quantise(x.astype(np.float64))
    got = oracle.pick(scales.numpy(), rows, columns)
    assert scales.numel() == oracle.scale_bytes(rows, columns) and np.array_equal(got, byte)
    fine = np.repeat(byte != 255, 32, 1)
    assert np.array_equal(codes.numpy()[fine], want[fine])
    with pytest.raises(ValueError):
        pack_mx8(torch.zeros(4, 100))


def test_norm_and_products_against_torch():
    rng = np.random.default_rng(2)
    x, r, g = rng.normal(0, 1, (5, 128)), rng.normal(0, 1, (5, 128)), rng.normal(1, 0.1, 128)
    s, n = oracle.norm(x, r, g, 1e-6)
    want = torch.nn.functional.rms_norm(torch.from_numpy(x + r), (128,), torch.from_numpy(g), 1e-6)
    assert np.allclose(n, want.numpy(), rtol=1e-12) and np.array_equal(s, x + r)
    w = rng.normal(0, 1, (64, 128))
    xs, ws = torch.from_numpy(x), torch.from_numpy(w)
    gate, up = xs @ ws[:32].T, xs @ ws[32:].T
    assert np.allclose(oracle.gated(x, w, "silu"), torch.nn.functional.silu(gate) * up, rtol=1e-9, atol=1e-12)
    assert np.allclose(oracle.gated(x, w, "gelu"), torch.nn.functional.gelu(gate, approximate="tanh") * up, rtol=1e-9,
                       atol=1e-9)
    assert np.allclose(oracle.proj(x, w, None), xs @ ws.T)
