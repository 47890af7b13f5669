"""ple_gated_mx8 and ple_proj_mx8 on the GPU against float64."""

import numpy as np
import pytest
import torch

import hashed_gram_embedding_gb300 as ple
from oracle import eight_bit as oracle

from _eight_bit import check_bf16, check_mx8, gated_off, packed, room, sum_off, untouched_scales
from _helpers import bits, bf16_values, dev_err_word

pytestmark = pytest.mark.gpu


def normal(rows, columns, seed, scale=1.0):
    return np.random.default_rng(seed).normal(0, scale, (rows, columns))


def f64(t):
    return bf16_values(bits(t)).reshape(t.shape)


def proj(x8, w8, t, n, residual=None):
    out = torch.full((t + 1, n), 7.0, dtype=torch.bfloat16, device="cuda")
    err = dev_err_word()
    ple.ple_proj_mx8(*x8, *w8, out[:t], residual=residual, dev_err=err)
    assert int(err.item()) == 0 and (out[t] == 7.0).all()
    return out[:t]


# tokens, columns, rows: one token, few, tiles of 16 to 256 and one more or less, rows and columns of every remainder
PROJ = [(1, 128, 1), (1, 256, 7), (1, 4096, 1024), (2, 384, 130), (3, 8192, 256), (8, 1152, 129), (15, 640, 255),
        (16, 2048, 128), (17, 128, 384), (31, 512, 8), (32, 896, 257), (33, 3200, 200), (48, 1024, 520), (63, 256, 1000),
        (64, 16384, 136), (65, 384, 96), (100, 2176, 333), (127, 1280, 64), (128, 640, 513), (129, 256, 250),
        (200, 4096, 128), (255, 512, 512), (256, 1024, 768), (257, 768, 100), (300, 384, 1025), (513, 1408, 384),
        (777, 2176, 500), (1025, 128, 2048), (2048, 512, 640)]


@pytest.mark.parametrize("t,e,n", PROJ)
def test_proj(t, e, n):
    x8, x = packed(normal(t, e, t))
    w8, w = packed(normal(n, e, e, e ** -0.5))
    got = proj(x8, w8, t, n)
    check_bf16(got, x @ w.T, sum_off(x, w), "proj")


@pytest.mark.parametrize("t,e,n", [(1, 512, 100), (40, 256, 129), (130, 384, 64), (600, 512, 777), (1024, 256, 512)])
@pytest.mark.parametrize("kind", ["apart", "wide", "itself", "odd", "eighth", "one row"])
def test_residual(t, e, n, kind):
    x8, x = packed(normal(t, e, 1))
    w8, w = packed(normal(n, e, 2, e ** -0.5))
    r = torch.from_numpy(normal(t, n, 3)).to(torch.bfloat16).cuda()
    want = oracle.proj(x, w, f64(r))
    off = sum_off(x, w) + 2.0 ** -23 * (np.abs(want) + np.abs(f64(r)))
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    if kind == "itself":
        out, given = r, r
    elif kind == "wide":
        given = torch.zeros((t, n + 24), dtype=torch.bfloat16, device="cuda")[:, 8:8 + n].copy_(r)
    elif kind == "odd":  # rows at addresses of two bytes
        given = torch.zeros(t * n + 1, dtype=torch.bfloat16, device="cuda")[1:].view(t, n).copy_(r)
        out = torch.zeros(t * n + 3, dtype=torch.bfloat16, device="cuda")[3:].view(t, n)
    elif kind == "eighth":  # of 8 bytes and no more
        given = torch.zeros(t * n + 4, dtype=torch.bfloat16, device="cuda")[4:].view(t, n).copy_(r)
        out = torch.zeros(t * n + 12, dtype=torch.bfloat16, device="cuda")[12:].view(t, n)
    elif kind == "one row":  # for all tokens, as a bias
        given = r[:1].expand(t, n)
        want = oracle.proj(x, w, f64(r[:1]))
        off = sum_off(x, w) + 2.0 ** -23 * (np.abs(want) + np.abs(f64(r[:1])))
    else:
        given = r
    ple.ple_proj_mx8(*x8, *w8, out, residual=given)
    check_bf16(out, want, off, kind)


GATED = [(1, 128, 128), (1, 2048, 512), (2, 256, 384), (5, 4096, 128), (8, 896, 256), (16, 512, 640), (17, 1152, 128),
         (32, 384, 256), (33, 2176, 128), (64, 256, 1024), (65, 640, 384), (127, 512, 128), (128, 1024, 256),
         (129, 128, 512), (200, 768, 384), (256, 512, 256), (257, 384, 128), (300, 2048, 640), (513, 256, 896),
         (777, 2176, 384), (1025, 512, 256), (2048, 384, 512)]


@pytest.mark.parametrize("t,c,i", GATED)
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated(t, c, i, name):
    x8, x = packed(normal(t, c, t))
    w8, w = packed(normal(2 * i, c, c, 1.5 * c ** -0.5))
    codes, scales = room(t, i)
    err = dev_err_word()
    ple.ple_gated_mx8(*x8, *w8, codes, scales, activation=name, dev_err=err)
    assert int(err.item()) == 0
    check_mx8(codes, scales, oracle.gated(x, w, name), gated_off(x, w, name), name)
    assert untouched_scales(scales, t, i)


@pytest.mark.parametrize("t", [1, 40, 200, 600])
def test_tokens_that_are_not_numbers_stay_alone(t):
    c, i, n = 384, 256, 200
    x = normal(t, c, 4)
    bad = sorted({0, t // 2, t - 1})
    x[bad[0], 3] = np.nan
    x[bad[-1], 200] = np.inf
    x[bad[len(bad) // 2], 64:96] = np.nan
    x8, xv = packed(x)
    w8, w = packed(normal(2 * i, c, 5, c ** -0.5))
    codes, scales = room(t, i)
    ple.ple_gated_mx8(*x8, *w8, codes, scales)
    want = oracle.gated(xv, w, "silu")
    want[bad] = np.nan
    check_mx8(codes, scales, want, gated_off(np.nan_to_num(xv), w, "silu"))
    w8, w = packed(normal(n, c, 6, c ** -0.5))
    got = f64(proj(x8, w8, t, n))
    want = xv @ w.T
    want[bad] = np.nan
    check_bf16(got, want, sum_off(np.nan_to_num(xv), w))


@pytest.mark.parametrize("t", [1, 70, 300])
def test_weight_rows_that_are_not_numbers_stay_alone(t):
    c, i = 256, 128
    w = normal(2 * i, c, 5, c ** -0.5)
    w[3, 5] = np.nan       # the gate's row 3
    w[i + 77, 100] = np.inf  # the other half's row 77
    w8, wv = packed(w)
    x8, x = packed(normal(t, c, 4))
    out = proj(x8, w8, t, 2 * i)
    want = x @ np.nan_to_num(wv).T
    want[:, [3, i + 77]] = np.nan
    check_bf16(out, want, sum_off(x, np.nan_to_num(wv)))
    codes, scales = room(t, i)
    ple.ple_gated_mx8(*x8, *w8, codes, scales)
    want = oracle.gated(x, np.nan_to_num(wv), "silu")
    want[:, [3, 77]] = np.nan
    check_mx8(codes, scales, want, gated_off(x, np.nan_to_num(wv), "silu"))


@pytest.mark.parametrize("t", [1, 33, 150, 400])
@pytest.mark.parametrize("low,high", [(-60, 60), (-120, -20), (40, 60)])
def test_values_of_any_size(t, low, high):
    # every block of columns, token and row with a power of its own: sums over terms far apart
    e, n = 512, 144
    rng = np.random.default_rng(t + low + 200)
    spread = lambda rows: 2.0 ** np.repeat(rng.integers(low, high, (rows, e // 32)), 32, 1)  # noqa: E731
    x8, x = packed(normal(t, e, 1) * spread(t))
    w8, w = packed(normal(n, e, 2) * spread(n))
    got = proj(x8, w8, t, n)
    # products below 2^-126 may lose bits, or all
    check_bf16(got, x @ w.T, sum_off(x, w) + e * 2.0 ** -126, "proj")


@pytest.mark.parametrize("t", [1, 64, 300])
def test_zeros(t):
    x8, x = packed(np.zeros((t, 256)))
    w8, w = packed(normal(256, 256, 2))
    assert (proj(x8, w8, t, 256) == 0).all()
    codes, scales = room(t, 128)
    ple.ple_gated_mx8(*x8, *w8, codes, scales)
    assert (codes & 0x7F == 0).all() and (oracle.pick(scales.cpu().numpy(), t, 128) == 0).all()


@pytest.mark.parametrize("t", [1, 60, 129, 700])
def test_same_call_same_bits(t):
    x8, _ = packed(normal(t, 2176, 1))
    w8, _ = packed(normal(640, 2176, 2, 0.02))
    first = [proj(x8, w8, t, 640).clone()]
    codes, scales = room(t, 320 // 128 * 128)
    w2 = packed(normal(512, 2176, 3, 0.02))[0]
    ple.ple_gated_mx8(*x8, *w2, codes, scales)
    first += [codes.clone(), scales.clone()]
    for _ in range(5):
        ple.ple_gated_mx8(*x8, *w2, codes, scales)
        assert all(torch.equal(a, b) for a, b in zip(first, (proj(x8, w8, t, 640), codes, scales)))


def test_a_token_does_not_depend_on_its_batch_far_beyond_rounding():
    # the kernels differ by how many tokens there are; each result is within its own bound of float64
    x = normal(600, 1024, 1)
    w8, w = packed(normal(384, 1024, 2, 1 / 32))
    for t in (1, 16, 17, 64, 65, 128, 129, 256, 257, 512, 600):
        x8, xv = packed(x[:t])
        check_bf16(proj(x8, w8, t, 384), xv @ w.T, sum_off(xv, w), str(t))


def test_refusals():
    x8, _ = packed(normal(4, 256, 1))
    w8, _ = packed(normal(256, 256, 2))
    out = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    codes, scales = room(4, 128)
    for args in ((x8[0][:, :128], x8[1], *w8, out), (x8[0], x8[1][:100], *w8, out), (*x8, w8[0].float(), w8[1], out),
                 (*x8, *w8, out[:3]), (*x8, *w8, out.float()), (*x8, *w8, out.t()), (x8[0].cpu(), x8[1], *w8, out)):
        with pytest.raises(ValueError):
            ple.ple_proj_mx8(*args)
    for kw in (dict(residual=out[:2]), dict(residual=out.float()), dict(dev_err=out)):
        with pytest.raises(ValueError):
            ple.ple_proj_mx8(*x8, *w8, out, **kw)
    for args in ((*x8, *w8, codes[:, :64], scales), (*x8, w8[0][:128], w8[1], codes, scales),
                 (*x8, *w8, codes[:3], scales), (*x8, *w8, codes, scales[:10])):
        with pytest.raises(ValueError):
            ple.ple_gated_mx8(*args)
    with pytest.raises(ValueError):
        ple.ple_gated_mx8(*x8, *w8, codes, scales, activation="relu")
    with pytest.raises(ple.PleError):
        ple.ple_gated_mx8(*x8, *w8, x8[0][:, :].view(-1)[:512].view(4, 128), scales)
    assert (codes == 0x5A).all() and (out == 0).all()


def test_no_tokens():
    x8, w8 = room(0, 256), packed(normal(256, 256, 2))[0]
    ple.ple_proj_mx8(*x8, *w8, torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"))
    ple.ple_gated_mx8(*x8, *w8, *room(0, 128))


def test_many_tokens():
    # codes of the gated result past 2^31 bytes, its values sampled
    t, c, i = 140_000, 128, 16384
    few = normal(1400, c, 1)
    (codes, scales), x = packed(few)
    big = codes.repeat(100, 1)
    byte = oracle.pick(scales.cpu().numpy(), 1400, c)
    big8 = big, torch.from_numpy(oracle.lay_out(np.tile(byte, (100, 1)), c, 0xFF)).cuda()
    w8, w = packed(normal(2 * i, c, 2, c ** -0.5))
    out = torch.empty((t, i), dtype=torch.uint8, device="cuda"), \
        torch.empty((oracle.scale_bytes(t, i),), dtype=torch.uint8, device="cuda")
    ple.ple_gated_mx8(*big8, *w8, *out)
    for lo in (0, 131_071, t - 2):
        at = np.arange(lo, lo + 2)
        pick = torch.from_numpy(np.stack([oracle.scale_at(r, np.arange(i // 32), i) for r in at])).cuda()
        laid = torch.from_numpy(oracle.lay_out(out[1][pick].cpu().numpy(), i)).cuda()
        rows = x[at % 1400]
        check_mx8(out[0][lo:lo + 2], laid, oracle.gated(rows, w, "silu"), gated_off(rows, w, "silu"))
    # and read by a product: 16384 columns
    n = 128
    w8, w = packed(normal(n, i, 3, i ** -0.5))
    y = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    ple.ple_proj_mx8(*out, *w8, y)
    for lo in (0, 131_071, t - 2):
        pick = np.stack([oracle.scale_at(r, np.arange(i // 32), i) for r in (lo, lo + 1)])
        rows = oracle.values(out[0][lo:lo + 2].cpu().numpy(), out[1][torch.from_numpy(pick).cuda()].cpu().numpy())
        check_bf16(y[lo:lo + 2], rows @ w.T, sum_off(rows, w))


def test_calls_at_once():
    """Both kernels of both calls on two streams, captured and not: nothing is shared."""
    cases = []
    for t in (1, 50, 300, 900):
        x8, _ = packed(normal(t, 640, t))
        w8, _ = packed(normal(1024, 640, t + 1, 0.04))
        codes, scales = room(t, 512)
        out = torch.zeros((t, 1024), dtype=torch.bfloat16, device="cuda")

        def run(x8=x8, w8=w8, codes=codes, scales=scales, out=out):
            ple.ple_gated_mx8(*x8, *w8, codes, scales)
            ple.ple_proj_mx8(*x8, *w8, out)

        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        cases.append((run, graph, (codes, scales, out)))
    want = []
    for run, _, outs in cases:
        run()
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(8):
        for i, (run, graph, outs) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                for o in outs:
                    o.zero_()
                if i % 2 == 0:
                    graph.replay()
                else:
                    run()
        torch.cuda.synchronize()
        for (_, _, outs), w in zip(cases, want):
            assert torch.equal(outs[0], w[0]) and torch.equal(outs[2], w[2])
            there = w[1] != 0xA5
            assert torch.equal(outs[1][there], w[1][there])
