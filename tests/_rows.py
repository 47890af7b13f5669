"""Checks of ple_kv_attention row by row, for cases of _four_bit.Batch.

Bounds. With u = 2^-8 (a bf16 has 8 significant bits), over any n elements of a row:
  * the result's rounding: u |want| at most;
  * roundings of weights, values and keys, 2^-11 (f16) at most where a kernel does them, independent from one
    position to the next: of weight and value 2^-11 / sqrt(3) each as a mean square, of a key's elements a
    score's error of 2^-11 / sqrt(3) scale sqrt(sum_d (q_d K_d)^2) in the exponent. (Weights are bf16, 2^-8,
    where few rows meet values of unusual size; `weights` says so.) Weights w_p that are off
    by independent parts r move an element by r sqrt(sum_p w_p^2 v_p^2). Four times that over n elements
    covers the spread of sums of as few as one position;
  * float32 arithmetic: 2^-16 of the largest value seen.
A whole output's rounding is that of its elements: uniform within half a step each, so its 2-norm is
sqrt(sum step^2 / 12); with the independent rest (squares add) it holds within 0.15 for a thousand elements
and more."""

import numpy as np

from _four_bit import oracle
from oracle.numerics import bf16_bits_to_f64

U = 2.0 ** -8
F16 = 2.0 ** -11
GROUP = 16


def reference(b, q, scale=None, causal=True, window=0):
    """float64 results [T, H, D] of q (bf16 bits [T, H, D]) over b's cache, and what the bounds are made of:
    spread [T, H, D] = sqrt(sum_p w_p^2 v_p^2), keyed [T, H, D] the same with a key's error beside the value's,
    sqrt(sum_p w_p^2 v_p^2 (1 + reach_p^2)), reach_p = scale |q K_p| (2-norm over d), and top [T, H] the largest
    |v| seen."""
    T, H, D = q.shape
    G = H // b.kv_heads
    scale = D ** -0.5 if scale is None else scale
    want, spread, keyed = (np.zeros((T, H, D)) for _ in range(3))
    top = np.zeros((T, H))
    x = bf16_bits_to_f64(q)
    for r in range(len(b.lens)):
        t0, t1, n = int(b.qsl[r]), int(b.qsl[r + 1]), int(b.lens[r])
        if t0 == t1 or n <= 0:
            continue
        rows = [oracle.read(b.cache, b.table, r, p, D) for p in range(n)]
        there = np.array([v is not None for v in rows])
        kv = np.array([np.zeros((2, b.kv_heads, D)) if v is None else v for v in rows])
        at = np.arange(n)
        for t in range(t0, t1):
            last = n - (t1 - t) if causal else n - 1
            seen = there & (at <= last)
            if window:
                seen &= at > last - window
            if not seen.any():
                continue
            for h in range(H):
                K, V = kv[seen, 0, h // G], kv[seen, 1, h // G]
                s = K @ x[t, h] * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                want[t, h] = w @ V
                spread[t, h] = np.sqrt(w ** 2 @ V ** 2)
                reach = scale ** 2 * ((x[t, h] * K) ** 2).sum(1)
                keyed[t, h] = np.sqrt((w ** 2 * (1 + reach)) @ V ** 2)
                top[t, h] = np.abs(V).max()
    return want, spread, keyed, top


def faults(got, want, spread, keyed, top, weights=F16):
    """What is out of bounds: a list of texts, empty for a right result."""
    found = []
    if not np.isfinite(got).all():
        return ["not finite"]
    err = got - want
    part = np.sqrt(((weights * spread) ** 2 + (F16 * keyed) ** 2) / 3)  # of an element, as a mean square
    D = got.shape[-1]
    for n in (GROUP, D):
        def norm(a):
            return np.sqrt((a.reshape(a.shape[:2] + (-1, n)) ** 2).sum(-1))
        bound = U * norm(want) + 4 * norm(part) + 2.0 ** -16 * np.sqrt(n) * top[..., None]
        bad = norm(err) > bound
        if bad.any():
            t, h, i = np.argwhere(bad)[0]
            found.append(f"{int(bad.sum())} of {bad.size} stretches of {n} elements, the first at token {t}, head {h}, "
                         f"element {i * n}: {norm(err)[t, h, i]:.3g}, bound {bound[t, h, i]:.3g}")
    step = np.where(want != 0, 2.0 ** (np.floor(np.log2(np.abs(np.where(want != 0, want, 1.0)))) - 7), 0.0)
    # case by case the largest values lead, so each row counts by its own size
    unit = np.maximum(np.sqrt((want ** 2).mean(-1, keepdims=True)), 1e-300)
    rounded = np.sqrt(((step / unit) ** 2).sum() / 12)
    rest = np.sqrt(((part / unit) ** 2).sum())
    total = np.sqrt(((err / unit) ** 2).sum())
    single = 2.0 ** -16 * np.sqrt(((top[..., None] / unit) ** 2).sum() * D)
    limit = 1.15 * np.sqrt(rounded ** 2 + rest ** 2 + single ** 2)
    if got.size >= 1000 and total > limit:
        found.append(f"the whole: {total:.4g}, bound {limit:.4g}")
    return found
