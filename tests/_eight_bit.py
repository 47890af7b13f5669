"""Cases and tolerances of the 8-bit step's tests.

A kernel's float32 value v' of a result v (float64) is off by at most `off`.
Quantised, it is off by half a step of e4m3 more: 2^-4 of itself, or, below
e4m3's least normal value, half of 2^-9 in units of the block's power of two,
which is at most the block's largest value / 224 (a smaller one would not have
held it), or 2^-127."""

import numpy as np
import torch

from hashed_gram_embedding_gb300 import pack_mx8
from oracle import eight_bit as oracle

from _helpers import bits, bf16_values

GARBAGE = 0xFF  # scale bytes of rows that do not exist: NaN, if they were used


def packed(x, device="cuda"):
    """8-bit tensor of float64 rows: (codes, scales) on the device, float64 values."""
    codes, scales = pack_mx8(torch.from_numpy(np.asarray(x, np.float32)))
    byte = oracle.pick(scales.numpy(), *x.shape)
    return ((codes.to(device), torch.from_numpy(oracle.lay_out(byte, x.shape[1], GARBAGE)).to(device)),
            oracle.values(codes.numpy(), byte))


def room(rows, columns, device="cuda"):
    """An 8-bit result's codes and scales, filled with a pattern."""
    return (torch.full((rows, columns), 0x5A, dtype=torch.uint8, device=device),
            torch.full((oracle.scale_bytes(rows, columns),), 0xA5, dtype=torch.uint8, device=device))


def untouched_scales(scales, rows, columns):
    """True if the bytes of rows that do not exist are as `room` left them."""
    s = scales.cpu().numpy()
    there = np.zeros(s.shape, bool)
    there[oracle._places(rows, columns)] = True
    return bool((s[~there] == 0xA5).all())


def check_mx8(codes, scales, want, off, what=""):
    """codes and scales (on the device) against float64 rows `want`, each float32 value off by `off` at most."""
    rows, columns = want.shape
    byte = oracle.pick(scales.cpu().numpy(), rows, columns).astype(np.int64)
    got = oracle.values(codes.cpu().numpy(), byte.astype(np.uint8))
    off = np.broadcast_to(off, want.shape)
    blocks = lambda a: a.reshape(rows, columns // 32, 32)  # noqa: E731
    bad = ~np.isfinite(blocks(want)).all(2)
    assert np.array_equal(byte == 255, bad), f"{what}: NaN blocks"
    assert np.isnan(blocks(got)[bad]).all(), f"{what}: values of NaN blocks"
    fine = np.repeat(~bad, 32, 1)
    want, off = np.where(fine, want, 0.0), np.where(fine, off, 0.0)
    top, slack = blocks(np.abs(want)).max(2), blocks(off).max(2)
    holds = 448.0 * 2.0 ** (byte - 127.0) >= top - slack
    least = (byte == 0) | (448.0 * 2.0 ** (byte - 128.0) < top + slack)
    assert (holds & least)[~bad].all(), f"{what}: scales"
    unit = np.maximum((top + slack) / 224.0, 2.0 ** -127)
    tol = 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * np.repeat(unit, 32, 1) + off * (1 + 2.0 ** -4)
    err = np.where(fine, np.abs(got - want), 0.0)
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.size} off, worst {np.max(err - tol)}"


def sum_off(x, w):
    """How far a float32 sum of len(x[0]) products may be off, in whatever
    order: n - 1 additions, each rounded by 2^-24 of a partial sum that is at
    most the sum of the magnitudes (twice that where additions cut off instead
    of rounding)."""
    return x.shape[1] * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T)


def check_bf16(out, want, off, what=""):
    got = bf16_values(bits(out)) if isinstance(out, torch.Tensor) else out
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN"
    fine = ~np.isnan(want)
    err = np.abs(got[fine] - want[fine])
    tol = 2.0 ** -8 * np.abs(want[fine]) + (np.broadcast_to(off, want.shape)[fine]) * (1 + 2.0 ** -8)
    assert (err <= tol).all(), f"{what}: {int((err > tol).sum())} of {err.size} off, worst {np.max(err - tol)}"


def gated_off(x, w, name):
    """How far float32's h may be off: both sums, the activation's slope (at
    most 1.13 for either), and 2^-18 for what it rounds itself."""
    inner = w.shape[0] // 2
    off = sum_off(x, w)
    og, ou = off[:, :inner], off[:, inner:]
    g, u = x @ w[:inner].T, x @ w[inner:].T
    h = oracle.activation(g, name)
    return 1.13 * og * (np.abs(u) + ou) + np.abs(h) * ou + 2.0 ** -18 * np.abs(h * u)
