"""ple_norm_mx8 and ple_mx8_read on the GPU against float64."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from oracle import eight_bit as oracle

from _eight_bit import check_bf16, check_mx8, packed, room, untouched_scales
from _helpers import bits, bf16_values

pytestmark = pytest.mark.gpu

EPS = 1e-6
# the float32 norm: 45 additions in the longest chain of a sum of squares
# (halved by the root) and 6 roundings more, below 2^-18
OFF = 2.0 ** -18


def rows(t, c, seed=0, scale=1.0):
    x = torch.from_numpy(np.random.default_rng(seed).normal(0, 1, (t, c)).astype(np.float32))
    return (x * scale).to(torch.bfloat16)


def f64(t):
    return bf16_values(bits(t)).reshape(t.shape)


def run(x, residual, gamma, eps=EPS, sum_out=True):
    t, c = x.shape
    codes, scales = room(t, c)
    out = torch.full((t, c), 3.0, dtype=torch.bfloat16, device="cuda") if sum_out else None
    dev = lambda a: None if a is None else a.cuda()  # noqa: E731
    ple.ple_norm_mx8(dev(x), dev(gamma), codes, scales, residual=dev(residual), sum_out=out, eps=eps)
    return codes, scales, out


def check(x, residual, gamma, got, eps=EPS):
    codes, scales, out = got
    s, n = oracle.norm(f64(x), None if residual is None else f64(residual), None if gamma is None else f64(gamma), eps)
    check_mx8(codes, scales, n, OFF * np.abs(n), "norm")
    assert untouched_scales(scales, *x.shape)
    if out is not None:
        check_bf16(out, s, 2.0 ** -24 * np.abs(s), "sum")


@pytest.mark.parametrize("t,c", [(1, 128), (1, 4096), (2, 4224), (3, 16384), (127, 256), (128, 2176), (129, 640),
                                 (257, 1152), (31, 8192), (5, 3968)])
@pytest.mark.parametrize("residual", [False, True])
def test_sizes(t, c, residual):
    x, r, g = rows(t, c), rows(t, c, 1, 3.0) if residual else None, rows(1, c, 2)[0]
    check(x, r, g, run(x, r, g))


def test_without_gamma_or_sum():
    x, r = rows(9, 512), rows(9, 512, 1)
    check(x, r, None, run(x, r, None, sum_out=False))
    check(x, None, None, run(x, None, None))


def test_strides_and_places():
    t, c = 33, 384
    wide = rows(t, 3 * c).cuda()
    x, r = wide[:, :c], wide[:, c:2 * c]
    want = [a.clone() for a in run(x.cpu(), r.cpu(), None)]
    for where in ("apart", "x", "residual"):
        wide2 = wide.clone()
        x, r = wide2[:, :c], wide2[:, c:2 * c]
        out = {"apart": wide2[:, 2 * c:], "x": x, "residual": r}[where]
        codes, scales = room(t, c)
        ple.ple_norm_mx8(x, None, codes, scales, residual=r, sum_out=out)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and torch.equal(out, want[2])
        for i, name in enumerate(("x", "residual", "apart")):
            if name != where:
                assert torch.equal(wide2[:, i * c:(i + 1) * c], wide[:, i * c:(i + 1) * c])


@pytest.mark.parametrize("exponent", [-133, -126, -70, -40, 40, 62, 100, 127])
@pytest.mark.parametrize("eps", [1e-6, 1e-38])
def test_rows_of_any_size(exponent, eps):
    # bf16's least and largest: squares leave float32 on both sides
    t, c = 4, 256
    rng = np.random.default_rng(exponent + 200)
    x = rng.uniform(0.25, 1, (t, c)) * rng.choice([-1, 1], (t, c)) * 2.0 ** exponent
    x = torch.from_numpy(x).to(torch.float32).to(torch.bfloat16)
    g = rows(1, c, 2)[0]
    check(x, None, g, run(x, None, g, eps), float(np.float32(eps)))


def test_rows_of_any_size_side_by_side():
    # narrow rows share a CTA, and only some of them leave float32
    for c in (128, 512, 640, 1408):
        x = rows(23, c)
        x[1::3] *= 2.0 ** 100
        x[2::7] *= 2.0 ** -110
        x[5] = 0
        g = rows(1, c, 2)[0]
        eps = float(np.float32(1e-30))
        check(x, None, g, run(x, None, g, eps), eps)


def test_many_narrow_rows():
    # CTAs that stay: more than four rows each, in place, odd in number
    t, c = 20_011, 384
    x, r = rows(t, c), rows(t, c, 1)
    want = run(x, r, None)
    check(x, r, None, want)
    d = x.cuda()
    codes, scales = room(t, c)
    ple.ple_norm_mx8(d, None, codes, scales, residual=r.cuda(), sum_out=d)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1]) and torch.equal(d, want[2])


def test_rows_that_are_not_numbers():
    t, c = 6, 384
    x = rows(t, c)
    x[1, 7] = float("nan")
    x[2] = 0
    x[3, 200] = float("inf")
    codes, scales, out = run(x, None, None)
    value = torch.empty((t, c), dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(codes, scales, value)
    v = f64(value)
    assert np.isnan(v[1]).all() and (v[2] == 0).all()
    assert np.isnan(v[3, 192:224]).all()  # inf / inf in its block
    assert (v[3, :192] == 0).all() and (v[3, 224:] == 0).all()  # and x / inf beside it
    # rows beside them are as without them
    y = rows(t, c)
    again = run(y, None, None)
    for r in (0, 4, 5):
        assert torch.equal(codes[r], again[0][r])
    assert np.array_equal(f64(out), f64(x), equal_nan=True)


def test_one_large_channel():
    # a block of tiny values beside a channel that sets the norm
    x = rows(3, 256) * 1e-3
    x[:, 40] = 1000.0
    g = torch.ones(256, dtype=torch.bfloat16)
    check(x, None, g, run(x, None, g))


@pytest.mark.parametrize("t,c", [(1, 128), (130, 384), (77, 4096)])
def test_read(t, c):
    x = np.random.default_rng(t).normal(0, 1, (t, c)) * 2.0 ** np.random.default_rng(1).integers(-60, 60, (t, 1))
    (codes, scales), want = packed(x)
    out = torch.full((t + 1, c), 7.0, dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(codes, scales, out[:t])
    assert np.array_equal(f64(out[:t]), want)  # exact
    assert (out[t] == 7.0).all()


def test_read_to_16_bytes():
    (codes, scales), want = packed(np.random.default_rng(0).normal(0, 1, (33, 256)))
    out = torch.zeros(33 * 256 + 8, dtype=torch.bfloat16, device="cuda")
    moved = torch.zeros(33 * 256 + 16, dtype=torch.uint8, device="cuda")[16:].view(33, 256).copy_(codes)
    ple.ple_mx8_read(moved, scales, out[8:].view(33, 256))
    assert np.array_equal(f64(out[8:].view(33, 256)), want) and (out[:8] == 0).all()


def test_read_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8).view(2, 128).repeat(128, 1)
    byte = np.arange(256, dtype=np.uint8)[:, None].repeat(4, 1)
    scales = torch.from_numpy(oracle.lay_out(byte, 128)).cuda()
    out = torch.empty((256, 128), dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(codes.cuda(), scales, out)
    want = oracle.values(codes.numpy(), byte)
    with np.errstate(over="ignore"):
        rounded = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)
    assert np.array_equal(f64(out), f64(rounded), equal_nan=True)


def test_refusals():
    x = rows(4, 256).cuda()
    codes, scales = room(4, 256)
    bad = [dict(x=x.float()), dict(x=x[:3]), dict(x=x.cpu()), dict(x=x.t()), dict(gamma=x[0, :128]),
           dict(gamma=x.float()[0]), dict(codes=codes[:, :128]), dict(codes=codes.float()), dict(scales=scales[:500]),
           dict(scales=scales.view(1, -1)), dict(residual=x[:2]), dict(sum_out=x.float()), dict(codes=codes.cpu())]
    for kw in bad:
        args = dict(x=x, gamma=None, codes=codes, scales=scales) | kw
        with pytest.raises(ValueError):
            ple.ple_norm_mx8(**args)
    with pytest.raises(ple.PleError):
        ple.ple_norm_mx8(x, None, codes, scales, eps=0.0)
    with pytest.raises(ValueError):
        ple.ple_mx8_read(codes, scales, x[:2])
    with pytest.raises(ple.PleError):  # the sum over other rows of x
        ple.ple_norm_mx8(x[:3], None, codes[:3], scales, sum_out=x.view(-1)[8:8 + 768].view(3, 256))
    assert (codes == 0x5A).all() and (scales == 0xA5).all()


def test_no_tokens():
    codes, scales = room(0, 256)
    ple.ple_norm_mx8(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), None, codes, scales)
    ple.ple_mx8_read(codes, scales, torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"))


def test_many_rows():
    # codes past 2^31 bytes: rows sampled
    t, c = 140_000, 16384
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((t // 100, c), generator=g, device="cuda").to(torch.bfloat16).repeat(100, 1)
    codes = torch.empty((t, c), dtype=torch.uint8, device="cuda")
    scales = torch.empty((oracle.scale_bytes(t, c),), dtype=torch.uint8, device="cuda")
    ple.ple_norm_mx8(x, None, codes, scales)
    for lo in (0, 131_000, t - 3):  # 131072 * 16384 = 2^31
        at = slice(lo, lo + 3)
        few = run(x[at].cpu(), None, None)
        assert torch.equal(codes[at], few[0])
        blocks = np.arange(c // 32)
        for i in range(3):
            got = scales[torch.from_numpy(oracle.scale_at(lo + i, blocks, c)).cuda()].cpu().numpy()
            assert np.array_equal(got, oracle.pick(few[1].cpu().numpy(), 3, c)[i])
    value = torch.empty((t, c), dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(codes, scales, value)
    small = torch.empty((3, c), dtype=torch.bfloat16, device="cuda")
    ple.ple_mx8_read(*run(x[-3:].cpu(), None, None)[:2], small)
    assert torch.equal(value[-3:], small)
