"""The 4-bit attention step in plain NumPy: the paged key/value cache in 4
bits, attention over it, and the projection with 4-bit weights (the formulas
stated in include/ple.h at ple_kv_append, ple_kv_attention, ple_proj_w4).

The cache's stored bytes follow from float32 operations rounded one by one,
so append restates those in np.float32 and its bytes are compared for
equality; attention and the projection are float64 over the stored values.
"""


import numpy as np

from .numerics import bf16_bits_to_f64 as bf16_to_f64, f64_to_bf16_bits as f64_to_bf16

BLOCK = 16


def _bf16(x):
    """float32 values -> bf16 bits, round to nearest even (NaN stays NaN)."""
    return f64_to_bf16(np.asarray(x, np.float32).astype(np.float64))


def _f32(bits):
    return bf16_to_f64(bits).astype(np.float32)


def rotate(x, cos_sin, position, interleaved):
    """x float32 [..., D], rotated by the table's row: the pairs' products and
    sums each rounded to float32."""
    rot = cos_sin.shape[1]
    cos, sin = cos_sin[position, :rot // 2], cos_sin[position, rot // 2:]
    y = x.copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def quantise(row):
    """codes uint8 [D], (scale, offset) bf16 bits of one float32 row."""
    with np.errstate(all="ignore"):
        lo, hi = np.min(row), np.max(row)  # NaN if any is
        pair = np.array([_bf16((hi - lo) * np.float32(1 / 15)), _bf16(lo)], np.uint16).reshape(2)
        scale, offset = _f32(pair)
        codes = np.zeros(row.shape, np.uint8)
        if scale > 0:
            y = np.rint((row - offset) / scale)
            codes = np.clip(np.where(np.isnan(y), 0, y), 0, 15).astype(np.uint8)
    return codes, pair


def block_parts(block, dim):
    """Views of one block's bytes: K codes, V codes, K pairs, V pairs."""
    n = BLOCK * dim // 2
    pairs = block[2 * n:].view(np.uint16).reshape(2, BLOCK, 2)
    return block[:n].reshape(BLOCK, dim // 2), block[n:2 * n].reshape(BLOCK, dim // 2), pairs[0], pairs[1]


def place(cache, block_table, r, p):
    """(page, sub-block, slot) of position p of request r, or None outside the cache."""
    page_size = cache.shape[2] * BLOCK
    if p < 0 or p // page_size >= block_table.shape[1]:
        return None
    page = int(block_table[r, p // page_size])
    if not 0 <= page < cache.shape[0]:
        return None
    return page, p % page_size // BLOCK, p % BLOCK


def tokens(qsl, kv_lens, num_tokens):
    """(token, request, position) of every token that is not padding."""
    for r in range(len(qsl) - 1):
        for t in range(int(qsl[r]), int(qsl[r + 1])):
            yield t, r, int(kv_lens[r]) - (int(qsl[r + 1]) - t)


def append(q, k, v, cos_sin, cache, block_table, qsl, kv_lens, positions=None, interleaved=False):
    """q, k, v bf16 bits [T, heads, D]; the cache (uint8) is updated in place.
    Returns q_out as bf16 bits."""
    out = np.zeros_like(q)
    dim = k.shape[2]
    for t, r, p in tokens(qsl, kv_lens, q.shape[0]):
        at = p if positions is None else int(positions[t])
        if cos_sin is not None and not 0 <= at < cos_sin.shape[0]:
            continue
        qt, kt, vt = _f32(q[t]), _f32(k[t]), _f32(v[t])
        if cos_sin is not None:
            qt, kt = rotate(qt, cos_sin, at, interleaved), rotate(kt, cos_sin, at, interleaved)
        out[t] = _bf16(qt)
        where = place(cache, block_table, r, p)
        if where is None:
            continue
        page, sub, slot = where
        for h in range(k.shape[1]):
            kc, vc, kp, vp = block_parts(cache[page, h, sub], dim)
            for row, code, pair in ((kt[h], kc, kp), (vt[h], vc, vp)):
                c, pair[slot] = quantise(row)
                code[slot] = c[0::2] | (c[1::2] << 4)
    return out


def read(cache, block_table, r, p, dim):
    """Keys and values [heads, D] in float64 at position p of request r, or None."""
    where = place(cache, block_table, r, p)
    if where is None:
        return None
    page, sub, slot = where
    out = np.zeros((2, cache.shape[1], dim))
    for h in range(cache.shape[1]):
        parts = block_parts(cache[page, h, sub], dim)
        for i in (0, 1):
            code, pair = parts[i][slot], bf16_to_f64(parts[2 + i][slot])
            with np.errstate(all="ignore"):
                out[i, h, 0::2] = (code & 15) * pair[0] + pair[1]
                out[i, h, 1::2] = (code >> 4) * pair[0] + pair[1]
    return out


def attention(q, cache, block_table, qsl, kv_lens, scale, causal=True, window=0):
    """q bf16 bits [T, H, D] -> float64 [T, H, D], and for every row the sum
    over d of |q_d| times the largest |K_pd| that it sees, and the largest
    |V| that it sees (what a bound on the result's error is made of)."""
    T, H, D = q.shape
    G = H // cache.shape[1]
    out, kmax, vmax = np.zeros((T, H, D)), np.zeros((T, H)), np.zeros((T, H))
    seen = {}
    for t, r, p in tokens(qsl, kv_lens, T):
        if r not in seen:
            rows = [read(cache, block_table, r, x, D) for x in range(int(kv_lens[r]))]
            seen = {r: (np.array([x is not None for x in rows], bool),
                        np.array([np.zeros((2, cache.shape[1], D)) if x is None else x for x in rows]))}
        there, kv = seen[r]
        last = p if causal else int(kv_lens[r]) - 1
        first = max(0, last - window + 1) if window else 0
        at = [x for x in range(first, last + 1) if there[x]]
        if not at:
            continue
        for h in range(H):
            K, V = kv[at, 0, h // G], kv[at, 1, h // G]
            x = bf16_to_f64(q[t, h])
            s = K @ x * scale
            w = np.exp(s - s.max())
            out[t, h] = w @ V / w.sum()
            kmax[t, h] = (np.abs(K) @ np.abs(x)).max() * scale
            vmax[t, h] = np.abs(V).max()
    return out, kmax, vmax


def proj_w4(x, codes, scales, zeros, group):
    """x bf16 bits [T, E], codes uint8 [N, E/2] -> float64 [T, N], and the sums
    of the absolute products."""
    N, half = codes.shape
    W = np.empty((N, 2 * half))
    W[:, 0::2], W[:, 1::2] = codes & 15, codes >> 4
    col = np.arange(2 * half) // group
    W = (W - (8 if zeros is None else zeros[:, col].astype(np.float64))) * bf16_to_f64(scales)[:, col]
    X = bf16_to_f64(x)
    return X @ W.T, np.abs(X) @ np.abs(W).T
