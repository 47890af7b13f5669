"""ple_proj_mx8 and ple_gated_mx8: their float32 sums, at sizes that reach every
kernel, tile and way of sharing the columns, several tiles a pair of CTAs and
tokens past its first group of 4096; the residual in every place."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from hashed_gram_embedding_gb300 import pack_mx8
from oracle import eight_bit as oracle

from _eight_bit import check_mx8, untouched_scales
from _helpers import dev_err_word
from _mx8_sums import GATED, PROJ, check_exact, check_sums, exact_operands, lay_out, left_over, random_operands

pytestmark = pytest.mark.gpu

PLACES = ("apart", "itself", "wide", "odd", "odd rows")


def placed(r, kind):
    """The residual in a place, and where the result goes."""
    t, n = r.shape
    new = lambda k, at: torch.zeros(t * n + k, dtype=torch.bfloat16, device="cuda")[at:at + t * n].view(t, n)  # noqa: E731
    if kind == "itself":
        r = r.clone()
        return r, r
    if kind == "wide":
        return torch.zeros((t, n + 24), dtype=torch.bfloat16, device="cuda")[:, 8:8 + n].copy_(r), new(0, 0)
    if kind == "odd":  # both begin at addresses of two bytes
        return new(1, 1).copy_(r), new(3, 3)
    if kind == "odd rows":  # an odd distance apart
        return torch.zeros((t, n + 1 + n % 2), dtype=torch.bfloat16, device="cuda")[:, :n].copy_(r), new(8, 8)
    return r.clone(), new(0, 0)


@pytest.mark.parametrize("t,e,n", [c[:3] for c in PROJ])
def test_proj_exact(t, e, n):
    x8, x, w8, w = exact_operands(t, e, n, seed=t + n, device="cuda")
    want = x @ w.T
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    err = dev_err_word()
    ple.ple_proj_mx8(*x8, *w8, out, dev_err=err)
    check_exact(out, want, torch.zeros_like(out))
    # the row that all tokens share, as a bias
    bias = left_over(want[:1])
    ple.ple_proj_mx8(*x8, *w8, out, residual=bias.expand(t, n), dev_err=err)
    assert torch.equal(out, (want + bias.double()).float().to(torch.bfloat16))
    # what is left beside the sum's first bits, the residual in every place
    r = left_over(want)
    for kind in PLACES:
        given, to = placed(r, kind)
        ple.ple_proj_mx8(*x8, *w8, to, residual=given, dev_err=err)
        check_exact(to, want, r)
    assert int(err.item()) == 0


@pytest.mark.parametrize("t,e,n", [c[:3] for c in PROJ])
def test_proj_random(t, e, n):
    x8, x, w8, w = random_operands(pack_mx8, t, e, n, seed=t + n, device="cuda")
    want = x @ w.T
    r = left_over(want)
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    ple.ple_proj_mx8(*x8, *w8, out, residual=r)
    check_sums(out, want, r, e)


@pytest.mark.parametrize("t,c,i", [k[:3] for k in GATED])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_exact(t, c, i, name):
    """Both sums are exact, so that h is off by the activation's roundings
    alone: 11 of 2^-24, and gelu's t by 5 |t| of them."""
    unit = -round(np.log2(75 * c ** 0.5))  # gates of about 1
    x8, x, w8, w = exact_operands(t, c, 2 * i, seed=t + i, device="cuda", unit=unit)
    codes = torch.full((t, i), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.full((oracle.scale_bytes(t, i),), 0xA5, dtype=torch.uint8, device="cuda")
    err = dev_err_word()
    ple.ple_gated_mx8(*x8, *w8, codes, scales, activation=name, dev_err=err)
    assert int(err.item()) == 0
    g, u = (x @ w[:i].T).cpu().numpy(), (x @ w[i:].T).cpu().numpy()
    assert np.array_equal(g.astype(np.float32), g)
    turn = g if name == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    small = np.exp(-np.abs(turn))
    want = g * np.where(turn >= 0, 1.0, small) / (1.0 + small) * u
    off = np.abs(want) * (11 + (0 if name == "silu" else 5 * np.abs(turn))) * 2.0 ** -24 + np.abs(g * u) * 2.0 ** -148 + 2.0 ** -149
    check_mx8(codes, scales, want, off, name)
    assert untouched_scales(scales, t, i)


@pytest.mark.parametrize("t,e,n", [(1, 4096, 300), (50, 4096, 300), (100, 4096, 300), (200, 4096, 300), (1500, 4096, 1000)])
def test_proj_whole_numbers_to_24_bits(t, e, n):
    """Sums of whole numbers, all of one sign, that grow past 2^23: float32 holds each on the way."""
    g = torch.Generator(device="cuda").manual_seed(t)

    def tensor(rows, low):
        whole = torch.randint(low, 16, (rows, e), generator=g, device="cuda") * \
            2 ** torch.randint(0, 5, (rows, e), generator=g, device="cuda")
        codes = whole.float().to(torch.float8_e4m3fn).view(torch.uint8)
        return (codes, lay_out(torch.full((rows, e // 32), 127, dtype=torch.uint8, device="cuda"))), whole.double()

    (x8, x), (w8, w) = tensor(t, 1), tensor(n, 0)
    want = x @ w.T
    assert 2 ** 22.8 < float(want.max()) < 2 ** 24
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    r = left_over(want)
    ple.ple_proj_mx8(*x8, *w8, out, residual=r)
    check_exact(out, want, r)
