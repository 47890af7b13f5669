"""Products of 8-bit tensors whose float32 sums are known to the last bit, and
bounds that 16-bit sums do not pass; works on any device.

Exact sums. Codes are whole numbers of -15 .. 15, the powers of a row's and a
weight row's blocks of columns cancel up to a power for the row and one for the
weight row, so that all products of a result are whole numbers of one unit,
225 at most: sums of up to 65536 of them stay below 2^24 units, and each
partial sum is exact in float32 whatever the order. What a residual of
-bf16(sum) leaves is then known exactly, and its bf16 as well."""

import numpy as np
import torch

# tokens, columns, rows, the tile of single CTAs that takes it (0: pairs of CTAs), CTAs that share the columns
# on 152 SMs with 76 pairs; checked against the library's rule without a GPU
PROJ = [
    (1, 16384, 4096, 32, 8), (30, 4096, 20000, 32, 1), (7, 1152, 2400, 32, 2), (32, 512, 129, 32, 1),
    (64, 16384, 136, 64, 8), (50, 2176, 20001, 64, 1), (48, 4096, 5000, 64, 4),
    (128, 8192, 513, 128, 4), (100, 1024, 19501, 128, 1), (77, 4096, 8200, 128, 2),
    (203, 16384, 4096, 256, 4), (200, 2176, 500, 256, 4), (200, 2176, 501, 256, 4), (777, 2176, 500, 256, 4),
    (777, 2176, 501, 256, 4), (512, 4096, 4096, 256, 2), (257, 8192, 2045, 256, 4),
    (1023, 2048, 8195, 0, 0), (4500, 256, 2501, 0, 0), (4500, 384, 2500, 0, 0), (2048, 16384, 4096, 0, 0),
    (8192, 4096, 4096, 0, 0), (2000, 4096, 5003, 0, 0), (9000, 128, 130, 0, 0),
]
GATED = [
    (1, 4096, 16384, 16, 2), (16, 384, 20096, 16, 1), (16, 8192, 1024, 16, 8), (3, 1152, 512, 16, 2), (32, 4096, 640, 32, 8), (20, 512, 20096, 32, 1),
    (64, 4096, 16384, 128, 1), (112, 4096, 4096, 128, 4), (40, 1024, 2048, 128, 2), (128, 16384, 256, 128, 4),
    (80, 2048, 8192, 0, 0), (777, 2176, 5504, 0, 0), (4500, 384, 1280, 0, 0), (2048, 4096, 4736, 0, 0),
    (300, 16384, 384, 0, 0),
]


def lay_out(byte):
    """Scale bytes uint8 [R, C / 32] in the library's order; 255 where no row is."""
    rows, blocks = byte.shape
    whole = torch.full((-(-rows // 128) * 128, blocks), 255, dtype=torch.uint8, device=byte.device)
    whole[:rows] = byte
    return whole.view(-1, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _tensor(rows, powers, g):
    """(codes, scales) and float64 values; powers int [rows, C / 32]."""
    whole = torch.randint(-15, 16, (rows, powers.shape[1] * 32), generator=g, device=powers.device).float()
    codes = whole.to(torch.float8_e4m3fn).view(torch.uint8)
    byte = (powers + 127).to(torch.uint8)
    return (codes, lay_out(byte)), whole.double() * torch.exp2(powers.double()).repeat_interleave(32, 1)


def exact_operands(tokens, columns, rows, seed=0, device="cpu", unit=0):
    """x and w as 8-bit tensors and their values; sums are whole numbers of
    2^unit times a power for the row and one for the weight row."""
    g = torch.Generator(device=device).manual_seed(seed)
    some = lambda n, m, low, high: torch.randint(low, high + 1, (n, m), generator=g, device=device)  # noqa: E731
    block = some(1, columns // 32, -6, 6)
    x8, x = _tensor(tokens, block + some(tokens, 1, -2, 2) + unit, g)
    w8, w = _tensor(rows, some(rows, 1, -2, 2) - block, g)
    return x8, x, w8, w


def random_operands(pack, tokens, columns, rows, seed=0, device="cpu"):
    """Normal x and w, quantised, and their values."""
    g = torch.Generator(device=device).manual_seed(seed)
    out = []
    for n, size in ((tokens, 1.0), (rows, columns ** -0.5)):
        codes, scales = pack(torch.randn(n, columns, generator=g, device=device) * size)
        byte = scales.view(-1, columns // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, columns // 32)[:n]
        power = torch.exp2(byte.double() - 127).repeat_interleave(32, 1)
        out += [(codes, scales), codes.view(torch.float8_e4m3fn).double() * power]
    return out


def left_over(want):
    """What is added to a sum so that its low bits stay: -bf16(want)."""
    return (-want).to(torch.float32).to(torch.bfloat16)


def check_exact(out, want, residual):
    """out is bf16(want + residual), all of it exact in float32."""
    rest = want + residual.double()
    assert torch.equal(rest.float().double(), rest)
    expect = rest.float().to(torch.bfloat16)
    bad = int((out.double() != expect.double()).sum())
    assert bad == 0, f"{bad} of {out.numel()} sums are not float32's"


def check_sums(out, want, residual, columns):
    """The 2-norm of the float32 sums' error. An addition of 32 columns'
    products is off by less than a unit in the last place, 2^-23 of a sum that
    is by the 2-norm at most the whole one; out's own rounding, of a rest below
    2^-9 of the sum, by 2^-17 of that."""
    err = out.double() - (want + residual.double())
    limit = (columns / 32 * 2.0 ** -23 + 2.0 ** -17) * float(want.square().mean().sqrt())
    rms = float(err.square().mean().sqrt())
    assert rms <= limit, f"rms {rms}, allowed {limit}"
