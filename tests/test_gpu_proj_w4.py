"""ple_proj_w4 on the GPU against float64. Bound of an element: the result's
rounding, 2^-8 relative (bf16 has 8 significant bits), and float32 sums whose terms the kernel may shift by
up to 144 code steps before it takes the shift out again (a code of at most 7
steps from its zero point meets the product as 128 + code): 16 roundings of
2^-24 (tensor-core sums in blocks, then a few joins) of 21 times the sum of
absolute products is below 2^-15 of that sum."""

import numpy as np
import pytest
import torch

from hashed_gram_embedding_gb300 import _lib

from _four_bit import bits, oracle
from _helpers import bf16_values

pytestmark = pytest.mark.gpu


def weight(N, E, group, with_zeros, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (N, E // 2), dtype=np.uint8)
    scales = torch.from_numpy(rng.uniform(0.002, 0.02, (N, E // group)).astype(np.float32)).to(torch.bfloat16)
    zeros = rng.integers(0, 16, (N, E // group)).astype(np.uint8) if with_zeros else None
    return codes, scales, zeros


def project(x, codes, scales, zeros, stream=None):
    out = torch.full((x.shape[0], codes.shape[0]), 7.0, dtype=torch.bfloat16, device="cuda")
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    _lib.ple_proj_w4(x, torch.from_numpy(codes).cuda(), scales.cuda(), out,
                     zeros=None if zeros is None else torch.from_numpy(zeros).cuda(), stream=stream)
    torch.cuda.synchronize()
    return out


def check(out, x, codes, scales, zeros, group):
    want, total = oracle.proj_w4(bits(x), codes, bits(scales), zeros, group)
    err = np.abs(bf16_values(bits(out)) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * total + 1e-30).all(), (err - 2.0 ** -8 * np.abs(want)).max()


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 150])
@pytest.mark.parametrize("E,group", [(32, 32), (128, 128), (320, 64), (1056, 32), (1024, 128), (2432, 64)])
@pytest.mark.parametrize("with_zeros", [False, True])
def test_against_float64(T, E, group, with_zeros):
    N = 8 * T + 37 if T < 20 else 129
    codes, scales, zeros = weight(N, E, group, with_zeros, seed=T + E)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    check(project(x.cuda(), codes, scales, zeros), x, codes, scales, zeros, group)


# many rows: every way the columns are shared out between CTAs, and none
@pytest.mark.parametrize("T,N,E,group", [(16, 14601, 160, 32), (17, 5000, 96, 32), (24, 4870, 2176, 128), (32, 9001, 1088, 64),
                                         (33, 700, 4096, 128), (64, 2500, 832, 64), (48, 9999, 640, 128), (64, 20001, 352, 32),
                                         (129, 6000, 1152, 128)])
@pytest.mark.parametrize("with_zeros", [False, True])
def test_many_rows(T, N, E, group, with_zeros):
    codes, scales, zeros = weight(N, E, group, with_zeros, seed=N + E)
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    check(project(x.cuda(), codes, scales, zeros), x, codes, scales, zeros, group)


@pytest.mark.parametrize("T", [20, 40])
@pytest.mark.parametrize("shift", [1, 3])
def test_many_rows_strided_and_unaligned(T, shift):
    """Rows of x far apart, scales and zero points at odd addresses, on another stream."""
    codes, scales, zeros = weight(5001, 512, 32, True, seed=T)
    wide = torch.randn(T, 512 + 64, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16)
    x = wide.cuda()[:, 32:32 + 512]
    held = torch.empty(scales.numel() + shift, dtype=torch.bfloat16, device="cuda")
    held_z = torch.empty(scales.numel() + shift, dtype=torch.uint8, device="cuda")
    s, z = held[shift:].view(scales.shape), held_z[shift:].view(scales.shape)
    s.copy_(scales)
    z.copy_(torch.from_numpy(zeros))
    out = torch.empty(T, 5001, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    _lib.ple_proj_w4(x, torch.from_numpy(codes).cuda(), s, out, zeros=z, stream=stream)
    torch.cuda.synchronize()
    check(out, wide[:, 32:32 + 512], codes, scales, zeros, 32)


@pytest.mark.parametrize("N", [1, 2, 15, 16, 17, 4099])
def test_output_sizes(N):
    codes, scales, zeros = weight(N, 512, 128, True, seed=N)
    x = torch.randn(3, 512, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16)
    check(project(x.cuda(), codes, scales, zeros), x, codes, scales, zeros, 128)


@pytest.mark.parametrize("mean", [0.0, 50.0])
def test_strided_rows_shifted_inputs_on_another_stream(mean):
    codes, scales, zeros = weight(300, 2048, 64, True, seed=9)
    wide = (torch.randn(12, 2048 + 64, generator=torch.Generator().manual_seed(3)) + mean).to(torch.bfloat16)
    x = wide[:, 32:2048 + 32]
    out = project(wide.cuda()[:, 32:2048 + 32], codes, scales, zeros, stream=torch.cuda.Stream())
    check(out, x, codes, scales, zeros, 64)
    again = project(wide.cuda()[:, 32:2048 + 32], codes, scales, zeros)
    assert torch.equal(again.view(torch.int16), out.view(torch.int16))


def test_values_that_are_not_finite_stay_in_their_row():
    codes, scales, zeros = weight(40, 256, 32, True, seed=21)
    x = torch.randn(5, 256, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    x[1, 7], x[3, 9] = float("nan"), float("inf")
    out = project(x.cuda(), codes, scales, zeros).cpu().float()
    assert out[1].isnan().all() and not torch.isfinite(out[3]).any()
    rest = [0, 2, 4]
    check(out[rest].to(torch.bfloat16), x[rest], codes, scales, zeros, 32)


def test_weight_past_32_bit_offsets():
    """Codes of 4.3 GB: the last rows start past 2^32 bytes."""
    N, E = 1_050_000, 8192
    codes = torch.zeros((N, E // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((N, E // 128), dtype=torch.bfloat16, device="cuda")
    c, s, _ = weight(16, E, 128, False, seed=33)
    codes[-16:], scales[-16:] = torch.from_numpy(c).cuda(), s.cuda()
    x = torch.randn(1, E, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16)
    out = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    _lib.ple_proj_w4(x.cuda(), codes, scales, out)
    torch.cuda.synchronize()
    check(out[:, -16:], x, c, s, None, 128)
    assert not out[:, :-16].any()
