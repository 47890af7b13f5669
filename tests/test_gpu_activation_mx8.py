"""ple_gated_mx8's activation, by itself: gates and factors whose sums are
exact, so that what is left is the activation's own error."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from _eight_bit import check_mx8, packed, room, untouched_scales

pytestmark = pytest.mark.gpu

GATES = (-1e13, -200.0, -108.0, -103.0, -95.0, -88.0, -87.0, -80.0, -60.0, -30.0, -14.0, -10.0, -9.5, -8.0, -5.0, -3.0,
         -1.0, -0.25, 0.0, 0.5, 2.0, 9.0, 30.0, 100.0, 200.0, 1e13)
FACTORS = (-100, -20, 0, 60, 110)  # powers of two of the other factor


def turns(g, name):
    return g if name == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)


def sigmoid(t):
    """Without cancelling on either side."""
    small = np.exp(-np.abs(t))
    return np.where(t >= 0, 1.0, small) / (1.0 + small)


def operands(tokens):
    """x [tokens, 128] and w [2 I, 128]: a gate is p_i + c_t q_i, near GATES[b]
    for the rows i of block b, the other factor v_i d_t 2^k."""
    rng = np.random.default_rng(tokens)
    blocks = [(g, min(k, 70 if abs(g) > 1e6 else k)) for g in GATES for k in FACTORS]  # h stays in float32
    blocks += [(1.0, 0)] * (-len(blocks) % 4)
    inner = 32 * len(blocks)
    x, w = np.zeros((tokens, 128)), np.zeros((2 * inner, 128))
    x[:, 0] = 1.0
    x[:, 1] = rng.integers(-15, 16, tokens) / 8.0
    x[:, 32] = rng.integers(8, 16, tokens) / 8.0
    for b, (g, k) in enumerate(blocks):
        at = slice(32 * b, 32 * b + 32)
        w[at, 0] = g
        w[at, 1] = rng.integers(-15, 16, 32) / 32.0 * max(1.0, 2.0 ** np.floor(np.log2(max(abs(g), 1.0))) / 64)
        w[inner:][at, 32] = rng.integers(8, 16, 32) / 8.0 * rng.choice([-1, 1], 32) * 2.0 ** k
    return x, w, inner


@pytest.mark.parametrize("tokens", [1, 13, 30, 100, 300, 1100])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activation(tokens, name):
    """h = g s(t) u, s(t) = 1 / (1 + exp(-t)), by float32 functions. Roundings,
    in units of 2^-24 of the result: exp 4 (2 units in the last place), the sum
    1, the quotient 4, two products 2, the exponent's t (nothing where it is g
    itself, else 5 of its value: two constants, three operations) 5 |t|. Where
    the exponential leaves float32's normal range it is off by 2^-148 at most."""
    x, w, inner = operands(tokens)
    (x8, xv), (w8, wv) = packed(x), packed(w)
    g, u = xv @ wv[:inner].T, xv @ wv[inner:].T
    assert np.array_equal(g.astype(np.float32), g) and np.array_equal(u.astype(np.float32), u)
    codes, scales = room(tokens, inner)
    ple.ple_gated_mx8(*x8, *w8, codes, scales, activation=name)
    t = turns(g, name)
    want = g * sigmoid(t) * u
    assert (np.abs(g * u) < 2.0 ** 127).all()
    off = np.abs(want) * (11 + (0 if name == "silu" else 5 * np.abs(t) * (t < 0))) * 2.0 ** -24
    off += np.abs(g * u) * 2.0 ** -148 + 2.0 ** -149
    check_mx8(codes, scales, want, off, name)
    assert untouched_scales(scales, tokens, inner)


@pytest.mark.parametrize("tokens", [1, 40, 300])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_infinite_gates(tokens, name):
    """Sums past float32's range: x / (1 + exp(-x)) of an infinity is itself, of
    minus infinity no number, and so is a block that holds either."""
    w = np.zeros((256, 128))
    w[:128, 0] = 1.0
    w[5, 0], w[40, 0] = 3e38, -3e38
    w[128:, 32] = 1.0
    x = np.zeros((tokens, 128))
    x[:, 0], x[:, 32] = 1.5, 1.0
    (x8, _), (w8, _) = packed(x), packed(w)
    codes, scales = room(tokens, 128)
    ple.ple_gated_mx8(*x8, *w8, codes, scales, activation=name)
    out = torch.empty((tokens, 128), dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(codes, scales, out)
    v = out.double().cpu().numpy()
    assert np.isnan(v[:, :64]).all()
    assert np.isfinite(v[:, 64:]).all() and (v[:, 64:] > 0.5).all()
