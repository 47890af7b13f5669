"""The 8-bit feed-forward step in plain NumPy, float64: the 8-bit format, the
norm with the residual's addition, the gated block and the projection (the
formulas stated in include/ple.h at ple_norm_mx8, ple_gated_mx8, ple_proj_mx8).

Codes and scales are decoded and quantised element by element from their
definition; scales travel as [rows, columns / 32] and `lay_out` / `pick`
move them to and from the library's order byte by byte.
"""

import numpy as np

from .numerics import E4M3_VALUES

BLOCK = 32
_MAGNITUDES = np.array([abs(float(v)) for v in E4M3_VALUES[:127]])  # codes 0 .. 126, increasing


def scale_bytes(rows, columns):
    return -(-rows // 128) * (columns // 128) * 512


def scale_at(r, j, columns):
    return ((r // 128) * (columns // 128) + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4


def _places(rows, columns):
    r, j = np.meshgrid(np.arange(rows), np.arange(columns // BLOCK), indexing="ij")
    return scale_at(r, j, columns)


def lay_out(byte, columns, fill=0):
    """Scale bytes [rows, columns / 32] in the library's order; `fill` where no row is."""
    out = np.full(scale_bytes(byte.shape[0], columns), fill, np.uint8)
    out[_places(byte.shape[0], columns)] = byte
    return out


def pick(scales, rows, columns):
    """Scale bytes [rows, columns / 32] out of the library's order."""
    return np.asarray(scales)[_places(rows, columns)]


def values(codes, byte):
    """float64 values of codes [R, C] and scale bytes [R, C / 32]."""
    power = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return np.asarray(E4M3_VALUES, np.float64)[codes] * np.repeat(power, BLOCK, 1)


def quantise(x):
    """codes and scale bytes of float64 rows, ties to the even code."""
    x = np.asarray(x, np.float64)
    rows, columns = x.shape
    codes = np.zeros(x.shape, np.uint8)
    byte = np.zeros((rows, columns // BLOCK), np.uint8)
    for r in range(rows):
        for j in range(columns // BLOCK):
            block = x[r, j * BLOCK:(j + 1) * BLOCK]
            top = np.max(np.abs(block))
            if not np.isfinite(top):
                byte[r, j] = 255
                continue
            b = 0
            while top > 448.0 * 2.0 ** (b - 127):
                b += 1
            byte[r, j] = b
            y = np.abs(block) / 2.0 ** (b - 127)
            above = np.clip(np.searchsorted(_MAGNITUDES, y), 1, 126)  # the code at or above
            low, high = _MAGNITUDES[above - 1], _MAGNITUDES[above]
            up = (y - low > high - y) | ((y - low == high - y) & (above % 2 == 0))
            codes[r, j * BLOCK:(j + 1) * BLOCK] = np.where(up, above, above - 1) | (np.signbit(block) * 128)
    return codes, byte


def norm(x, residual, gamma, eps):
    """(sum, normed rows) in float64."""
    s = x if residual is None else x + residual
    n = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps)
    return s, n if gamma is None else n * gamma


def activation(g, name):
    if name == "silu":
        return g / (1 + np.exp(-g))
    return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def gated(x, w, name):
    """act(x Wg^T) * (x Wu^T) of float64 values, w [2 I, C]."""
    inner = w.shape[0] // 2
    with np.errstate(all="ignore"):
        return activation(x @ w[:inner].T, name) * (x @ w[inner:].T)


def proj(x, w, residual):
    y = x @ w.T
    return y if residual is None else y + residual
