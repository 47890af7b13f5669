"""The products' tests find sums of fewer bits, and reach every kernel (no GPU)."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from hashed_gram_embedding_gb300 import build, pack_mx8

from _mx8_sums import GATED, PROJ, check_exact, check_sums, exact_operands, left_over, random_operands

T, E, N = 24, 4096, 40


def running(products, step, dtype):
    """A sum over the last axis that is rounded after every `step` products."""
    s = torch.zeros(products.shape[:-1])
    for part in products.split(step, -1):
        s = (s + part.sum(-1).float()).to(dtype).float()
    return s


def in_parts(products, parts, dtype):
    """The parts' sums rounded, then added."""
    n = products.shape[-1] // parts
    return sum(p.sum(-1).to(dtype).float() for p in products.split(n, -1))


SUMS = {
    "float32": lambda p: running(p, 32, torch.float32),
    "float32 parts": lambda p: in_parts(p, 8, torch.float32),
    "float16 after 128 columns": lambda p: running(p, 128, torch.float16),
    "bfloat16 after 128 columns": lambda p: running(p, 128, torch.bfloat16),
    "parts in float16": lambda p: in_parts(p, 8, torch.float16),
    "parts in bfloat16": lambda p: in_parts(p, 8, torch.bfloat16),
    "two parts in float16": lambda p: in_parts(p, 2, torch.float16),
    "a block less": lambda p: p[..., 32:].sum(-1).float(),
    "a block twice": lambda p: (p.sum(-1) + p[..., :32].sum(-1)).float(),
    "tf32 at the end": lambda p: (p.sum(-1).float().view(torch.int32) & -8192).view(torch.float32),
}


@pytest.mark.parametrize("how", SUMS)
@pytest.mark.parametrize("kind", ["exact", "random"])
def test_sums_of_fewer_bits_are_found(kind, how):
    if kind == "exact":
        _, x, _, w = exact_operands(T, E, N)
    else:
        _, x, _, w = random_operands(pack_mx8, T, E, N)
    want = x @ w.T
    residual = left_over(want)
    out = (SUMS[how](x[:, None, :] * w) + residual.float()).to(torch.bfloat16)
    check = (lambda: check_exact(out, want, residual)) if kind == "exact" else (lambda: check_sums(out, want, residual, E))
    if how.startswith("float32"):
        check()
    else:
        with pytest.raises(AssertionError):
            check()


def test_products_are_whole_numbers_of_a_unit():
    for t, e, n in ((5, 16384, 3), (3, 128, 4)):
        (_, x, _, w) = exact_operands(t, e, n, seed=e)
        unit = x.abs().amax(1, keepdim=True)  # (rows of x and w have powers of their own)
        assert (unit > 0).all()
        p = x[:, None, :] * w
        low = torch.where(p == 0, float("inf"), p.abs()).amin(-1, keepdim=True)
        power = torch.exp2(torch.floor(torch.log2(low)) - 8)
        assert (p / power == (p / power).round()).all() and (p.abs().sum(-1, keepdim=True) / low < 2 ** 24).all()


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    """The library's own rule, by itself."""
    at = tmp_path_factory.mktemp("rule")
    source = at / "rule.cpp"
    source.write_text('#include "mx8_rule.h"\n'
                      'extern "C" int tile(long long t, int e, int n, int gated, int sms, int pairs) {\n'
                      '  return ple::product_tile({t, e, n, gated != 0}, sms, [&] { return pairs; });\n}\n'
                      'extern "C" int parts(int tile, long long t, int e, int n, int sms) {\n'
                      '  return ple::few_parts(tile, (n + 127LL) / 128 * ((t + tile - 1) / tile), e / 128, sms);\n}\n')
    so = str(at / "rule.so")
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(source),
                    "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.tile.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 5
    lib.parts.argtypes = [ctypes.c_int, ctypes.c_longlong] + [ctypes.c_int] * 3
    return lib


@pytest.mark.parametrize("gated,cases", [(0, PROJ), (1, GATED)])
def test_shapes_reach_the_kernels_they_are_for(rule, gated, cases):
    for t, e, n, tile, parts in cases:
        got = rule.tile(t, e, n, gated, 152, 76)
        assert (got, rule.parts(got, t, e, n, 152) if got else 0) == (tile, parts), (t, e, n)
    # every tile, with columns shared out and not, and pairs with several tiles each, past the first 4096 tokens
    assert {c[3] for c in cases} == ({0, 16, 32, 128} if gated else {0, 32, 64, 128, 256})
    for tile in {c[3] for c in cases} - {0}:
        at = {c[4] for c in cases if c[3] == tile}
        assert (2 if tile == 256 else 1) in at and (4 if tile >= 128 else 8) in at, tile
    rows = 128 if gated else 256
    units = [(-(-t // 256) * -(-n // rows), t, n % rows) for t, e, n, tile, _ in cases if tile == 0]
    assert any(u > 2 * 76 for u, *_ in units) and any(u > 76 and t > 4096 for u, t, _ in units)
    if not gated:
        assert any(u > 2 * 76 and t > 4096 and odd for u, t, odd in units)
