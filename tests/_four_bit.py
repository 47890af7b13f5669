"""Cases of the 4-bit step's tests: a ragged batch with its paged cache, on
the host as NumPy (the oracle's side) and on the device."""

import numpy as np
import torch

from _helpers import bits, from_bits
from oracle import four_bit as oracle

NAN = 0x7FC1  # a bf16 NaN


class Batch:
    """queries[r] new tokens and lens[r] cached positions (these included) for
    each request; pages shuffled, every byte that no position uses garbage:
    random codes with NaN scales."""

    def __init__(self, queries, lens, heads, kv_heads, dim, page, seed=0, spare=3, pad=0, k_mean=1.0):
        self.rng = rng = np.random.default_rng(seed)
        self.queries, self.lens = list(queries), np.array(lens, np.int32)
        self.heads, self.kv_heads, self.dim, self.page = heads, kv_heads, dim, page
        self.qsl = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
        self.T = int(self.qsl[-1]) + pad
        need = [-(-max(int(n), 0) // page) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = rng.integers(0, self.pages, (len(lens), max(need + [1]) + 1)).astype(np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        sub = page // 16
        self.cache = rng.integers(0, 256, (self.pages, kv_heads, sub, 16 * (dim + 8)), dtype=np.uint8)
        self.cache[..., 16 * dim:] = np.full(64, NAN, np.uint16).view(np.uint8)
        self.mean = rng.normal(0, k_mean, (kv_heads, dim))
        for r, n in enumerate(lens):
            for p in range(int(n)):
                self.put(r, p, rng.normal(0, 1, (kv_heads, dim)) + self.mean, rng.normal(0, 1, (kv_heads, dim)))

    def put(self, r, p, k, v):
        page, sub, slot = oracle.place(self.cache, self.table, r, p)
        for h in range(self.kv_heads):
            kc, vc, kp, vp = oracle.block_parts(self.cache[page, h, sub], self.dim)
            for row, code, pair in ((k[h], kc, kp), (v[h], vc, vp)):
                c, pair[slot] = oracle.quantise(np.asarray(row, np.float32))
                code[slot] = c[0::2] | (c[1::2] << 4)

    def rows(self, heads, scale=1.0):
        """bf16 normal rows [T, heads, dim] on the host."""
        x = self.rng.normal(0, scale, (self.T, heads, self.dim)).astype(np.float32)
        return torch.from_numpy(x).to(torch.bfloat16)

    def device(self):
        return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda()
                     for a in (self.cache, self.table, self.qsl, self.lens))


def rotation_table(positions, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    angle = np.arange(positions)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


__all__ = ["Batch", "rotation_table", "bits", "from_bits", "oracle", "NAN"]
